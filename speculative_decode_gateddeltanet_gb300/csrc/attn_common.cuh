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

#include "gdnlong.h"

namespace gdnattn {

constexpr unsigned kFull = 0xffffffffu;
// the kernels' positions and row numbers are 32-bit, and run up to a block past a request's last
constexpr int kMaxIndex = INT32_MAX - 1023;

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// 16 bytes into shared memory, or zeros
__device__ __forceinline__ void copy16(float* to, const float* from, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from), "r"(valid ? 16 : 0) : "memory");
}

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

// of gdn_paged_attention: its host checks, and the parameters but for the work buffer
int check(const gdn_paged_attn_args* a);
Params params_of(const gdn_paged_attn_args* a);
void set_work(Params& p, int dtype, void* work);  // notes and partials, gdn_paged_attention_work_bytes

// whether a tensor map of 16-bit elements can have the stride of a dimension of n entries: it has 40 bits of bytes
inline bool map_stride(int64_t elements, int64_t n) { return n <= 1 || elements < int64_t(1) << 39; }

struct Nothing {};

// What a shared call has beside them.
struct SharedParams {
  int n_groups, key_align;  // a request's own keys begin at a multiple of key_align
  const int32_t *group_start, *prefix_len;
  float* lse;
  int64_t lse_row;
  // rows that take part in a prefix, which are ranked request by request:
  int n_ranks;        // the most that can
  float* dense;       // [2][n_ranks * H_q][d]: first parts over prefixes and over own keys, unnormalised
  int4* entries;      // [2][n_ranks * H_q]: a first part's maximum and sum, its block, and entry_word
  int* rank_row;      // [n_ranks] each rank's row, or -1
  int* count;         // ranks
};

struct Request {
  int ctx, n, row0;
  __device__ int flat() const { return 0; }
  __device__ int len() const { return ctx + n; }                   // its keys' end
  __device__ int last(int token) const { return ctx + token; }     // the last key that a row sees
};

// A line of a shared call: a request's rows over its own keys, or the rows of a group over its prefix.  Keys count from
// k0; the first `front` of them are the prefix's still.
struct Line {
  int ctx, n, row0;  // group: prefix - 1, the rows of all its requests, the rank of the first among all such rows
  int k0, front;
  int b;       // table row
  int prefix;  // request: tokens of its shared prefix; group: -1
  __device__ int flat() const { return prefix < 0; }
  __device__ int len() const { return prefix < 0 ? ctx + 1 : ctx + n; }
  __device__ int last(int token) const { return prefix < 0 ? ctx : ctx + token; }
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
// Called, not copied into each place: a launch's first time through its code is bound by fetching it, and the kernels'
// roles together fill the instruction cache.
static __device__ __noinline__ long long floor_sum(long long n, long long m, long long a, long long b) {
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

template <int kRows, int kKeys, typename R = Request>
struct Tiles {
  __device__ static int count(const Params& p, const R& r) { return (int)(((unsigned long long)r.n * p.G + kRows - 1) / kRows); }
  __device__ static int blocks(const Params& p, const R& r, int m) {
    if (r.flat()) return (int)((unsigned)r.ctx / kKeys) + 1;
    const long long last = min((long long)(m + 1) * kRows, (long long)r.n * p.G) - 1;
    const int token = last >> 31 ? (int)(last / p.G) : (int)quotient((uint32_t)last, p.by_G);
    return (int)((unsigned)(r.ctx + token) / kKeys) + 1;
  }
  // Units that a tile costs beside its key blocks, in the time of one: about 3 us from a tile's last product to the next
  // one's first on the tensor cores.  Measured (64-key blocks, 128-key blocks): 16 x 4 rows at d = 256 take 35.7 us with
  // 5, 39.2 with 3 or 4, 36.1 with 10; prompt chunks of up to 4096 485 with 3, 493 with 2, 516 with 1, 504 with 6; 256
  // ragged requests 172 with 3, 177 with 6.
  static constexpr int kExtra = kRows < 128 ? 0 : kKeys == 64 ? 5 : 3;
  __device__ static int extra(const Params& p, const Request&) { return kExtra; }
  // In a shared call (128-key blocks: requests' tiles, prefixes' tiles) 64 single tokens behind 32768 take 99.4 us with 5 and
  // 3, 106 with 3 and 3, 105 with 8 and 3; 16 requests of 4 tokens behind 8011 at d = 256 31.7 with 5 and 8, 34.0 with 5 and 5.
  __device__ static int extra(const Params& p, const Line& l) { return kExtra == 0 ? 0 : kKeys == 64 && l.flat() ? 8 : l.prefix > 0 ? 5 : kExtra; }
  // units of the tiles before m
  __device__ static long long before(const Params& p, const R& r, int m) {
    if (m == 0) return 0;
    if (r.flat()) return (long long)m * (blocks(p, r, 0) + extra(p, r));
    return (long long)m * (1 + extra(p, r)) + floor_sum(m, (long long)p.G * kKeys, kRows, (long long)p.G * r.ctx + kRows - 1);
  }
  // units of one kv head of the request
  __device__ static long long sum(const Params& p, const R& r) {
    if (r.n <= 0) return 0;
    const int M = count(p, r);
    return before(p, r, M - 1) + extra(p, r) + blocks(p, r, M - 1);
  }
};

// Every line of a shared call, from its lengths and groups in shared memory.
struct Lines {
  int B, G;            // requests, then groups: line v < B is request v's
  int most;            // rows of a request that takes part in a prefix
  const int* starts;   // [G + 1]
  const int* prefix;   // [G] tokens that the group's requests read together; 0: none
  const int* rows;     // [B + 1] rows before request b of those that take part in a prefix
  // the group that request b is in, or -1
  __device__ int group_of(int b) const {
    if (G == 0 || b < starts[0] || b >= starts[G]) return -1;
    int lo = 0, hi = G;  // starts[lo] <= b < starts[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (starts[mid] <= b) lo = mid;
      else hi = mid;
    }
    return lo;
  }
  // the request whose counted rows hold that rank
  __device__ int request_of(int rank) const {
    int lo = 0, hi = B;  // rows[lo] <= rank < rows[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (rows[mid] <= rank) lo = mid;
      else hi = mid;
    }
    return lo;
  }
  __device__ Line own(const Request& r, int b, int align, int L) const {
    const int k0 = L & -align;  // a power of two
    return {r.ctx - k0, r.n, r.row0, k0, L - k0, b, L};
  }
  __device__ Line own(const Request& r, int b, int align) const {
    const int g = r.n > 0 ? group_of(b) : -1, L = g >= 0 ? prefix[g] : 0;
    return own(r, b, align, r.ctx < L || r.n > most ? 0 : L);
  }
  __device__ Line group(int g, bool find = true) const {  // find: its table row too, which its units do not depend on
    if (prefix[g] == 0 || rows[starts[g + 1]] == rows[starts[g]]) return {0, 0, 0, 0, 0, 0, -1};
    const int first = rows[starts[g]];
    return {prefix[g] - 1, rows[starts[g + 1]] - first, first, 0, 0, find ? request_of(first) : 0, -1};
  }
  __device__ Line line(const Params& p, int v, int align) const { return v < B ? own(request(p, v), v, align) : group(v - B); }
  // rank of a line's token, where the line's rows have parts over a prefix and over their own keys
  __device__ int rank_of(const Line& l, int token) const { return (l.flat() ? l.row0 : rows[l.b]) + token; }
  // row of q and o of a line's token
  __device__ int row_of(const Params& p, const Line& l, int token) const {
    if (!l.flat()) return l.row0 + token;
    const int rank = l.row0 + token, b = request_of(rank);
    return (p.row_start ? p.row_start[b] : b * p.R) + rank - rows[b];
  }
};

// one block's walk over its units, tile by tile
template <int kRows, int kKeys, bool kShared = false>
struct Walk {
  using R = std::conditional_t<kShared, Line, Request>;
  using T = Tiles<kRows, kKeys, R>;
  R req;
  int b, h, m, tiles, left;  // b: request or line; left: units still to do
  int at;                    // the segment's first unit within its tile: the tile's own units come first
  int kb0, kb1, blocks;      // its key blocks, and how many the whole tile has

  __device__ void segment() {
    blocks = T::blocks(*p, req, m);
    const int extra = T::extra(*p, req), end = min(extra + blocks, at + left);
    kb0 = max(0, at - extra);
    kb1 = end - extra;
    if (kb1 <= kb0) left = 0;  // the block's part ends before the tile's first key block
  }
  __device__ bool done() const { return left <= 0; }
  __device__ void next() {
    left -= kb1 + T::extra(*p, req) - at;
    if (left <= 0) return;
    at = 0;
    if (++m == tiles) {
      m = 0;
      if (++h == p->H_kv) {
        h = 0;
        do {
          if constexpr (kShared) req = lines->line(*p, ++b, align);
          else req = request(*p, ++b);
        } while (req.n <= 0);
        tiles = T::count(*p, req);
      }
    }
    segment();
  }
  __device__ int table_row() const {
    if constexpr (kShared) return req.b;
    else return b;
  }
  __device__ int first_key() const {
    if constexpr (kShared) return req.k0;
    else return 0;
  }
  const Params* p;
  const Lines* lines;
  int align;
};

template <typename R>
struct StartOf {
  long long total;  // units of the call
  long long off;    // units from the first request's first to the block's first
  long long head;   // units of one kv head of that request
  R req;            // the request the block begins in
  int b, per;
};
using Start = StartOf<Request>;

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

// The most rows of a request that takes part in a prefix: with them a tile of tile_rows is not yet full.
__host__ __device__ constexpr int most_rows(int tile_rows, int G) { return (tile_rows - 1) / G; }

// Words of shared memory that a shared call's lines take.
constexpr int kMaxSharedB = 4096, kMaxGroups = 512;
constexpr int lines_words(int B, int n_groups) { return B + 3 * n_groups + 2; }
constexpr int kMaxLinesWords = lines_words(kMaxSharedB, kMaxGroups);

// What a call must save by sharing, in units of one block: the join of every row's parts.  Measured (tensor cores, shared
// and unshared): 16 requests of 1 row of 4 heads behind 2048 tokens (25 units a block unshared) 22.3 and 32.7 us, of 8 rows
// 31.9 and 29.8; 4 of 4 rows of 8 heads behind 8192 at d = 256 28.2 and 22.1; 16 behind 16384 38.9 and 64.7.
constexpr int kShareGain = 6;
// And what a request's tile of its own and the join cost beside the units that the division counts: 64 requests of 16 tokens
// of 4 heads behind 1000 tokens 98 us shared, 70 not; of 1 token 57 and 65.
constexpr int kJoinUnits = 4;
#ifdef GDN_TEST_HOOKS
constexpr bool kShareAlways = true;  // test builds: whatever it costs
#else
constexpr bool kShareAlways = false;
#endif

// find_start for the lines of a shared call.  at: lines_words of shared memory, filled here; scan:
// 3 * kThreads/32 words.  Where group_start does not rise within [0, B], or the counted rows pass 32 bits, no prefix is
// shared, and what is computed is the same.
//
// A request takes part in its group's prefix where its rows do not fill a tile: behind a full one K and V are read for 128
// rows at least already, and the join of two parts costs more than the rows' closer packing gives (4 prompts of 400 to 1000
// tokens behind 8192: 435 us shared, 330 not; 16 requests of 32 tokens of 4 heads behind 16384: 152 and 142, of 16 tokens 99
// and 128).  A group shares where that leaves fewer units in all, and all groups together save more than kShareGain.
template <int kRows, int kKeys, int kThreads>
__device__ __forceinline__ Lines find_lines(const Params& p, const SharedParams& sp, int min_units, int* at, long long* scan,
                                            StartOf<Line>* out) {
  using T = Tiles<kRows, kKeys, Line>;
  __shared__ unsigned long long gain;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int each = (p.B + kThreads - 1) / kThreads, b0 = tid * each, b1 = min(p.B, b0 + each);
  int* const saved = at;  // [G] units of a kv head that a group's requests leave out
  int* const starts = saved + sp.n_groups;
  int* const prefix = starts + sp.n_groups + 1;
  int* const rows = prefix + sp.n_groups;
  int why = 0, broken = 0;
  Request first = {0, 0, 0};
  int first_g = -1;  // the group whose prefix it may meet
  const int reads = sp.n_groups > 0 && tid <= sp.n_groups;
  int x = 0, y = 0, length = 0;  // on their way with the request's
  if (reads) {
    x = sp.group_start[tid];
    if (tid < sp.n_groups) {
      y = sp.group_start[tid + 1];
      length = sp.prefix_len[tid];
    }
  }
  if (b0 < b1) first = request(p, b0, &why);
  for (int g = tid; g <= sp.n_groups && sp.n_groups > 0; g += kThreads) {
    if (g != tid) {
      x = sp.group_start[g];
      if (g < sp.n_groups) {
        y = sp.group_start[g + 1];
        length = sp.prefix_len[g];
      }
    }
    starts[g] = x;
    if (g < sp.n_groups) {
      prefix[g] = max(length, 0);
      saved[g] = 0;
    }
    broken |= x < 0 || x > p.B || (g < sp.n_groups && x > y);
  }
  if (tid == 0) gain = 0;
  broken = __syncthreads_or(broken);
  if (broken && blockIdx.x == 0 && tid == 0 && p.status) atomicOr(p.status, GDN_STATUS_BAD_GROUP);
  Lines lines = {p.B, broken ? 0 : sp.n_groups, most_rows(kRows, p.G), starts, prefix, rows};
  // exclusive sum of x over the threads, and the whole sum
  auto sums = [&](long long x, long long* part, long long* total) {
    long long inc = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long v = __shfl_up_sync(kFull, inc, off);
      if (lane >= off) inc += v;
    }
    if (lane == 31) part[warp] = inc;
    __syncthreads();
    long long before = inc - x, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += part[w];
      all += part[w];
    }
    *total = all;
    return before;
  };
  if (lines.G > 0) {
    // rows of request b that may meet the prefix; what its own line then lacks goes to its group
    auto counted = [&](const Request& r, int b) {
      const int g = r.n > 0 ? lines.group_of(b) : -1;
      return g < 0 || prefix[g] == 0 || r.ctx < prefix[g] || r.n > lines.most ? -1 : g;
    };
    long long mine = 0, total;
    for (int b = b0; b < b1; ++b) {
      const Request r = b == b0 ? first : request(p, b, &why);
      const int g = counted(r, b);
      if (b == b0) first_g = g;
      if (g < 0) continue;
      mine += r.n;
      // at most one tile, as the request's rows do not fill it
      const Line l = lines.own(r, b, sp.key_align, prefix[g]);
      const int whole = T::blocks(p, lines.own(r, b, sp.key_align, 0), 0), own = T::blocks(p, l, 0);
      atomicAdd(&saved[g], min(whole - own - kJoinUnits, 1 << 18));  // 4096 of them stay below 2^31
    }
    long long before = sums(mine, scan, &total);
    if (total > min(p.max_rows, p.n_q_rows)) {  // rows that overlap, or too many for a tile's numbers
      lines.G = 0;  // uniform
    } else {
      for (int b = b0; b < b1; ++b) {
        rows[b] = (int)before;
        if (b == b0) {
          before += first_g >= 0 ? first.n : 0;
        } else {
          const Request r = request(p, b);
          before += counted(r, b) >= 0 ? r.n : 0;
        }
      }
      if (tid == 0) rows[p.B] = (int)total;
      __syncthreads();
      for (int g = tid; g < lines.G; g += kThreads) {
        const long long less = saved[g] - T::sum(p, lines.group(g, false));
        if (kShareAlways) continue;
        if (less > 0) atomicAdd(&gain, (unsigned long long)(less * p.H_kv));
        else prefix[g] = 0;
      }
      __syncthreads();
      if (!kShareAlways && gain <= (unsigned long long)kShareGain * p.n_blocks) lines.G = 0;
    }
  } else {
    for (int b = b0 + 1; b < b1; ++b) request(p, b, &why);
  }
  if (why && blockIdx.x == 0 && p.status) atomicOr(p.status, why);
  if (blockIdx.x == gridDim.x - 1) {  // for the join; this block has the least to do
    for (int b = b0; b < b1 && lines.G > 0; ++b) {
      const int n = rows[b + 1] - rows[b], row0 = n == 0 ? 0 : b == b0 ? first.row0 : request(p, b).row0;
      const bool shares = n > 0 && prefix[b == b0 ? first_g : lines.group_of(b)] > 0;
      for (int t = 0; t < n; ++t) sp.rank_row[rows[b] + t] = shares ? row0 + t : -1;
    }
    if (tid == 0) *sp.count = lines.G > 0 ? rows[p.B] : 0;
  }
  long long mine = 0, mine_g = 0, head = 0, total, total_g = 0;
  Line l = {};
  for (int b = b0; b < b1; ++b) {
    l = b == b0 ? lines.own(first, b, sp.key_align, lines.G > 0 && first_g >= 0 ? prefix[first_g] : 0)
                : lines.own(request(p, b), b, sp.key_align);
    head = T::sum(p, l);
    mine += p.H_kv * head;
  }
  const int each_g = (lines.G + kThreads - 1) / kThreads, g0 = tid * each_g, g1 = min(lines.G, g0 + each_g);
  for (int g = g0; g < g1; ++g) mine_g += p.H_kv * T::sum(p, lines.group(g, false));
  long long mine_at, g_at;
  {
    long long x = mine, y = mine_g;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long u = __shfl_up_sync(kFull, x, off), v = __shfl_up_sync(kFull, y, off);
      if (lane >= off) {
        x += u;
        y += v;
      }
    }
    long long* const part = scan + kThreads / 32;
    if (lane == 31) {
      part[warp] = x;
      part[kThreads / 32 + warp] = y;
    }
    __syncthreads();
    mine_at = x - mine;
    g_at = y - mine_g;
    total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) {
        mine_at += part[w];
        g_at += part[kThreads / 32 + w];
      }
      total += part[w];
      total_g += part[kThreads / 32 + w];
    }
    g_at += total;
  }
  total += total_g;
  const long long per = max(total >> 31 ? (total + p.n_blocks - 1) / p.n_blocks
                                        : (long long)(((uint32_t)total + (uint32_t)p.n_blocks - 1) / (uint32_t)p.n_blocks),
                            (long long)min_units);
  const long long want = per * blockIdx.x;
  if (tid == 0) {
    out->total = total;
    out->per = (int)min(per, (long long)INT32_MAX);
  }
  // one thread at most finds the block's first unit in its part, of requests or of groups
  const bool in_own = want >= mine_at && want < mine_at + mine, in_group = want >= g_at && want < g_at + mine_g;
  if (in_own || in_group) {
    long long off = want - (in_own ? mine_at : g_at);
    int v = in_own ? b0 : p.B + g0;
    if (in_group || each > 1) {
      for (;; ++v) {
        l = lines.line(p, v, sp.key_align);
        head = T::sum(p, l);
        if (off < p.H_kv * head) break;
        off -= p.H_kv * head;
      }
    }
    out->b = v;
    out->off = off;
    out->head = head;
    out->req = l;
  }
  __syncthreads();
  return lines;
}

template <int kRows, int kKeys, bool kShared, typename S>
__device__ __forceinline__ bool begin(Walk<kRows, kKeys, kShared>& w, const Params& p, const S& s) {
  using T = typename Walk<kRows, kKeys, kShared>::T;
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

// blocks after the segment's that share its tile
template <typename W, typename S>
__device__ __forceinline__ int followers_of(const W& w, const S& s) {
  return (w.blocks - w.kb1 + s.per - 1) / s.per;
}
// The note of a split tile at its first block: the blocks that follow this one
// in it, its request's first row, kv head and rows, and its first row's number.
template <int kRows, int kKeys, bool kShared, typename S>
__device__ __forceinline__ int4 note_of(const Walk<kRows, kKeys, kShared>& w, const S& s) {
  const int rows = (int)min((long long)kRows, (long long)w.req.n * w.p->G - (long long)w.m * kRows);
  return {followers_of(w, s), w.req.row0, w.h << 8 | rows, w.m * kRows};
}

// a rank's place among its kv head's in `dense` and `entries`: a tile's rows lie together.  Places over prefixes come first.
__device__ __forceinline__ size_t place_of(const Params& p, const SharedParams& sp, bool own, int rank, int kv_head, int g) {
  return ((size_t)(own ? p.H_kv + kv_head : kv_head) * sp.n_ranks + rank) * p.G + g;
}
// What a first part's entry says beside its maximum, sum and block: the blocks that follow, and its row in the tile.
__device__ __forceinline__ int entry_word(int followers, int row) { return followers | row << 16; }
constexpr float kLn2 = 0.693147180559945309f;

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
  __shared__ __align__(8) float sums[kCombineWarps][kD];  // two columns at once
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

// A shared call's join: the rows of split tiles whose requests take part in no prefix, and the ranked rows, which join the
// parts over their request's own keys and over its prefix.  Every block adds up the notes' rows, so that all of them share
// both kinds of rows evenly, however few tiles are split.  A row's parts are added in one order: the first own one, those of
// the blocks that follow, the prefix's first and its followers.  kTeam warps share a row's parts: four where rows are few,
// and a tile is cut into many parts, one where they are many.
constexpr int kMostBlocks = 4 * 32 * kCombineWarps;  // of an attention launch

template <typename T, int kD, int kRows, int kTeam>
__global__ void __launch_bounds__(32 * kCombineWarps) combine_shared(const Params p, const SharedParams sp) {
  constexpr int kPer = kD / 32, kBatch = 4, kRowsAtOnce = kCombineWarps / kTeam;
  __shared__ __align__(8) float sums[kTeam > 1 ? kTeam : 1][kTeam > 1 ? kD : 1];  // two columns at once
  __shared__ int tile_rows[kMostBlocks], warp_rows[kCombineWarps];  // rows of the split tiles before each block's
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, member = warp % kTeam, H_q = p.H_kv * p.G;
  auto load = [&](float (&v)[kPer], const float* src) {
#pragma unroll
    for (int c = 0; c < kPer / 2; ++c) {
      const float2 y = *reinterpret_cast<const float2*>(src + c * 64 + lane * 2);
      v[2 * c] = y.x;
      v[2 * c + 1] = y.y;
    }
  };
  // One row: its first parts in acc and x_pre with their maxima and sums, then f_own parts of the blocks behind own_block at
  // row own_row of their tile, and f_pre of the prefix.
  auto join = [&](int row, int head, float (&acc)[kPer], const float (&x_pre)[kPer], float2 s_own, float2 s_pre, int own_block, int own_row,
                  int f_own, int pre_block, int pre_row, int f_pre) {
    const int f = f_own + f_pre;
    auto part = [&](int i) {
      return partial(p, i < f_own ? own_block + 1 + i : pre_block + 1 + i - f_own, 0, kRows) + (size_t)(i < f_own ? own_row : pre_row) * kD;
    };
    auto stats = [&](int i) {
      return reinterpret_cast<const float2*>(partial(p, i < f_own ? own_block + 1 + i : pre_block + 1 + i - f_own, 0, kRows) +
                                             (size_t)kRows * kD)[i < f_own ? own_row : pre_row];
    };
    float top = fmaxf(s_own.x, s_pre.x);
    float2 s_lane = make_float2(-INFINITY, 0.f);  // of part `lane`: all of them in most calls
    if (f > 0) {
      if (lane < f) s_lane = stats(lane);
      float t = s_lane.x;
      for (int i = lane + 32; i < f; i += 32) t = fmaxf(t, stats(i).x);
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) t = fmaxf(t, __shfl_xor_sync(kFull, t, off));
      top = fmaxf(top, t);
    }
    const float base = top == -INFINITY ? 0.f : top, w_own = exp2f(s_own.x - base), w_pre = exp2f(s_pre.x - base);
    float sum = s_own.y * w_own + s_pre.y * w_pre;
#pragma unroll
    for (int c = 0; c < kPer; ++c) acc[c] = kTeam == 1 || member == 0 ? acc[c] * w_own + x_pre[c] * w_pre : 0.f;
    if (f > 0) {
      float t = s_lane.y * exp2f(s_lane.x - base);
      for (int i = lane + 32; i < f; i += 32) {
        const float2 st = stats(i);
        t += st.y * exp2f(st.x - base);
      }
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) t += __shfl_xor_sync(kFull, t, off);
      sum += t;
      for (int i0 = member; i0 < f; i0 += kTeam * kBatch) {
        float v[kBatch][kPer], weight[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const int i = min(i0 + j * kTeam, f - 1);
          load(v[j], part(i));
          const float mine = f <= 32 ? __shfl_sync(kFull, s_lane.x, i) : stats(i).x;
          weight[j] = i0 + j * kTeam < f ? exp2f(mine - base) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          if (i0 + j * kTeam >= f) break;
#pragma unroll
          for (int c = 0; c < kPer; ++c) acc[c] = fmaf(weight[j], v[j][c], acc[c]);
        }
      }
    }
    if constexpr (kTeam > 1) {
      if (f > 0) {  // the same for the row's warps, which are all the block's
#pragma unroll
        for (int c = 0; c < kPer / 2; ++c)
          *reinterpret_cast<float2*>(&sums[warp][c * 64 + lane * 2]) = make_float2(acc[2 * c], acc[2 * c + 1]);
        __syncthreads();
        if (member == 0) {
#pragma unroll
          for (int c = 0; c < kPer; ++c) {
#pragma unroll
            for (int w = 1; w < kTeam; ++w) acc[c] += sums[w][(c / 2) * 64 + lane * 2 + (c & 1)];
          }
        }
        __syncthreads();
      }
      if (member > 0) return;
    }
    const float inv = 1.f / sum;
    T* const dst = static_cast<T*>(p.o) + (int64_t)row * p.o_row + (int64_t)head * p.o_head + lane * 2;
#pragma unroll
    for (int c = 0; c < kPer / 2; ++c) {
      const float a = acc[2 * c] * inv, z = acc[2 * c + 1] * inv;
      if constexpr (sizeof(T) == 2) *reinterpret_cast<__nv_bfloat162*>(dst + c * 64) = __floats2bfloat162_rn(a, z);
      else *reinterpret_cast<float2*>(dst + c * 64) = make_float2(a, z);
    }
    if (sp.lse && lane == 0) sp.lse[(int64_t)row * sp.lse_row + head] = (base + log2f(sum)) * kLn2;
  };
  const int count = *sp.count;
  constexpr int kEach = kMostBlocks / (32 * kCombineWarps);
  int mine[kEach], rows_here = 0;
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int x = threadIdx.x * kEach + k;
    const int4 note = x < p.n_blocks ? p.notes[x] : make_int4(0, 0, 0, 0);
    mine[k] = note.x > 0 ? note.z & 255 : 0;
    rows_here += mine[k];
  }
  int inc = rows_here;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(kFull, inc, off);
    if (lane >= off) inc += v;
  }
  if (lane == 31) warp_rows[warp] = inc;
  __syncthreads();
  int before = inc - rows_here, of_tiles = 0;
#pragma unroll
  for (int i = 0; i < kCombineWarps; ++i) {
    if (i < warp) before += warp_rows[i];
    of_tiles += warp_rows[i];
  }
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    tile_rows[threadIdx.x * kEach + k] = before;
    before += mine[k];
  }
  __syncthreads();
  const long long items = of_tiles + (long long)count * H_q;
  // where a block gave up, a row's entry may be anything
  auto inside = [&](const int4& e) { return e.z >= 0 && e.z < p.n_blocks && (e.w & 0xffff) < p.n_blocks - e.z && (e.w >> 16 & 255) < kRows; };
  // the two kinds of rows are one loop's items, so that the join is compiled once
  for (long long item = (long long)blockIdx.x * kRowsAtOnce + warp / kTeam; item < items; item += (long long)gridDim.x * kRowsAtOnce) {
    int row, head;
    float acc[kPer], x_pre[kPer] = {};
    int4 own, pre;
    if (item < of_tiles) {
      int x_block = 0, hi = p.n_blocks;  // tile_rows[x_block] <= item < tile_rows[hi], the last such block
      while (hi - x_block > 1) {
        const int mid = (x_block + hi) >> 1;
        if (tile_rows[mid] <= item) x_block = mid;
        else hi = mid;
      }
      const int4 note = p.notes[x_block];
      const int in_tile = (int)item - tile_rows[x_block], at = note.w + in_tile, token = (int)quotient(at, p.by_G);
      row = note.y + token;
      head = (note.z >> 8) * p.G + at - token * p.G;
      const float* const first = partial(p, x_block, 1, kRows);
      const float2 s = reinterpret_cast<const float2*>(first + (size_t)kRows * kD)[in_tile];
      own = make_int4(__float_as_int(s.x), __float_as_int(s.y), x_block, entry_word(note.x, in_tile));
      pre = make_int4(__float_as_int(-INFINITY), 0, 0, 0);
      if (kTeam == 1 || member == 0) load(acc, first + (size_t)in_tile * kD);
    } else {
      const long long i = item - of_tiles;
      const int rank = i >> 31 ? (int)(i / H_q) : (int)((uint32_t)i / (uint32_t)H_q);
      head = (int)(i - (long long)rank * H_q);
      row = sp.rank_row[rank];
      if (row < 0) continue;
      const int h = (int)quotient(head, p.by_G);
      const size_t own_at = place_of(p, sp, true, rank, h, head - h * p.G), pre_at = place_of(p, sp, false, rank, h, head - h * p.G);
      own = sp.entries[own_at];
      pre = sp.entries[pre_at];
      if (kTeam == 1 || member == 0) {
        load(acc, sp.dense + own_at * kD);
        load(x_pre, sp.dense + pre_at * kD);
      }
      if (!inside(own) || !inside(pre)) continue;  // the same for the row's warps
    }
    join(row, head, acc, x_pre, make_float2(__int_as_float(own.x), __int_as_float(own.y)),
         make_float2(__int_as_float(pre.x), __int_as_float(pre.y)), own.z, own.w >> 16 & 255, own.w & 0xffff, pre.z, pre.w >> 16 & 255,
         pre.w & 0xffff);
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

// A team of four warps a row where rows are so few that the GPU holds them all at once.
template <typename T, int kD, int kRows>
int launch_combine_shared(const Params& p, const SharedParams& sp, cudaStream_t st) {
  const long long rows = (long long)p.n_q_rows * p.H_kv * p.G;
  const dim3 block(32 * kCombineWarps);
  // no row is an item twice
  auto grid = [&](long long blocks) { return dim3((unsigned)(blocks < 152 * 16 ? blocks : 152 * 16)); };
  if (rows <= 152 * 16) return launch(combine_shared<T, kD, kRows, kCombineWarps>, grid(rows), block, 0, st, p, sp);
  return launch(combine_shared<T, kD, kRows, 1>, grid((rows + kCombineWarps - 1) / kCombineWarps), block, 0, st, p, sp);
}

}  // namespace gdnattn
