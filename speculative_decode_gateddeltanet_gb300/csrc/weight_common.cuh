// What the kernels of gdn_attn_weight share: parameters, the division of the work over blocks, and the writing of weights.
//
//   got[j] = sum over kv heads h, rows (t, g) with ctx + t >= j of 2^(scale log2(e) q[t, g].K[j, h] - log2(e) lse[t, g])
//
// Units.  Keys are cut into blocks of kKeys, a kv head's rows into tiles of `tokens` tokens by `heads` query heads (`parts`
//   tiles cover a token's G heads where G does not fit one).  A unit is one (key block, kv head, tile): one product and one
//   exponential an entry.  A key block needs the tiles from its first key's row on:
//     m0(kb) = parts * max(0, floor((kb kKeys - ctx) / tokens))
//   A run of tiles of one key block and head costs kRun units more: its K, and tiles that the diagonal crosses.
// Division.  All units of a call form one line, request by request, key block by key block, head by head, so that a key
//   block's sum over heads and rows stays in one block's registers; block i takes units [i per, (i+1) per).  A request's
//   units up to a key block are a floor sum (attn_common.cuh), so each block finds its part by itself.
// Join.  Where a key block's units lie in several blocks, the first of them leaves a partial in slot 1 and a note, each
//   other one in slot 0; join_kernel adds them in block order.  No sum depends on timing.
#pragma once
#include "attn_common.cuh"

namespace gdnattn {

struct WeightParams {
  Params p;  // its lines, q and K; o, V and the attention's work are unused
  float scale, keep;
  int fresh;
  const float* lse;
  int64_t lse_row;
  const int32_t *first, *position;
  float* weight;
  int32_t* born;
  int tokens, heads, parts;  // of a tile: tokens * heads rows
  Div by_heads, by_parts;
  int* notes;       // [n_blocks] blocks that follow in a key block that a block begins and does not end
  int* slots;       // [n_blocks][kKeys] its keys' slots, kNewSlot added for tokens that start anew, or -1
  float* partials;  // [n_blocks][2][kKeys]
};

// floor_sum where the numbers leave room: its divisions in 32 bits.  (With this and floor_sum called, and the next request
// found without them, the bf16 kernel's code is 82 KB in place of 152: 16 x 4 rows at d = 256 take 17.9 us, not 19.7, ragged
// single steps of 128 requests 67.4, not 69.3.)
static __device__ __noinline__ long long weight_floor_sum(int n, int m, int a, long long b) {
  if (((long long)n * (a > m ? a : m) + b) >> 31) return floor_sum(n, m, a, b);
  long long s = 0;
  uint32_t N = n, M = m, A = a, C = (uint32_t)b;
  while (N > 0) {
    if (A >= M) {
      const uint32_t q = A / M;
      s += (long long)N * (N - 1) / 2 * q;
      A -= q * M;
    }
    if (C >= M) {
      const uint32_t q = C / M;
      s += (long long)N * q;
      C -= q * M;
    }
    const uint32_t y = A * N + C;
    if (y < M) break;
    N = y / M;
    C = y - N * M;
    const uint32_t t = M;
    M = A;
    A = t;
  }
  return s;
}

struct WeightRequest {
  int ctx, n, row0, first;
  int kb0, kb1;  // key blocks: from the first index that takes weight to the last token
  int M;         // tiles of a head
};

template <int kKeys>
struct WeightUnits {
  // 8192 tokens at d = 64 take 220 us, with 2 226, 1 236, 0 264; at d = 128 258, with 2 257, 1 260, 0 280; prompts of 1500 to
  // 4096 tokens 79, with 2 80, 1 82, 0 90; single steps the same.
  static constexpr int kRun = kKeys == 128 ? 4 : 0;
  __device__ static WeightRequest request(const WeightParams& w, int b, int* why = nullptr) {
    const Request r = gdnattn::request(w.p, b, why);
    WeightRequest x = {r.ctx, r.n, r.row0, 0, 0, 0, 0};
    if (r.n <= 0) return x;
    x.first = w.first ? max(w.first[b], 0) : 0;
    const int len = r.ctx + r.n;
    x.kb0 = x.first / kKeys;
    x.kb1 = x.first < len ? (int)((unsigned)(len - 1) / kKeys) + 1 : x.kb0;
    x.M = (r.n + w.tokens - 1) / w.tokens * w.parts;
    return x;
  }
  // first tile that sees key block kb
  __device__ static int m0(const WeightParams& w, const WeightRequest& r, int kb) {
    const int past = kb * kKeys - r.ctx;
    return past > 0 ? past / w.tokens * w.parts : 0;
  }
  // units of one head in key blocks [0, kb)
  __device__ static long long before(const WeightParams& w, const WeightRequest& r, int kb) {
    const int K1 = r.ctx / kKeys + 1;  // the first block whose first key is not a cached token's, and m0 > 0 at most from there
    long long s = (long long)kb * (r.M + kRun);
    if (kb > K1) s -= w.parts * weight_floor_sum(kb - K1, w.tokens, kKeys, (long long)K1 * kKeys - r.ctx);
    return s;
  }
  // units of one head of the request
  __device__ static long long sum(const WeightParams& w, const WeightRequest& r) {
    return r.kb1 > r.kb0 ? before(w, r, r.kb1) - before(w, r, r.kb0) : 0;
  }
};

struct WeightStart {
  long long total, per, off;  // units of the call, of a block, and from the request's first to the block's first
  WeightRequest req;
  int b;
};

// Every thread of the block calls this; all get the block's first unit.  scan: kThreads/32 words of shared memory.
template <int kKeys, int kThreads>
__device__ __forceinline__ void find_weight_start(const WeightParams& w, long long* scan, WeightStart* out) {
  using U = WeightUnits<kKeys>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, B = w.p.B, n_blocks = w.p.n_blocks;
  const int each = (B + kThreads - 1) / kThreads, b0 = threadIdx.x * each, b1 = min(B, b0 + each);
  long long mine = 0;
  WeightRequest req = {};
  int why = 0;
  for (int b = b0; b < b1; ++b) {
    req = U::request(w, b, &why);
    mine += w.p.H_kv * U::sum(w, req);
  }
  if (why && blockIdx.x == 0 && w.p.status) atomicOr(w.p.status, why);
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
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) before += scan[i];
    total += scan[i];
  }
  const long long at = before + inc - mine;
  const long long per = max(U::kRun + 1ll, total >> 31 ? (total + n_blocks - 1) / n_blocks
                                             : (long long)(((uint32_t)total + (uint32_t)n_blocks - 1) / (uint32_t)n_blocks));
  const long long want = per * blockIdx.x;
  if (threadIdx.x == 0) {
    out->total = total;
    out->per = per;
  }
  if (want >= at && want < at + mine) {  // one thread at most
    long long off = want - at;
    int b = b0;
    if (each > 1) {
      for (;; ++b) {
        req = U::request(w, b);
        const long long s = w.p.H_kv * U::sum(w, req);
        if (off < s) break;
        off -= s;
      }
    }
    out->b = b;
    out->off = off;
    out->req = req;
  }
  __syncthreads();
}

// a block's walk over its units
template <int kKeys>
struct WeightWalk {
  using U = WeightUnits<kKeys>;
  const WeightParams* w;
  WeightRequest req;
  int b, kb, h, m, low;  // low: m0 of kb
  int skip;              // the run's units before its tiles that are this block's
  long long left;        // units still to do, these among them
  bool whole;            // the block has its key block from its first unit

  __device__ bool begin(const WeightParams& params, const WeightStart& s) {
    w = &params;
    const long long first = s.per * blockIdx.x;
    left = max(0ll, min(s.per, s.total - first));
    if (left <= 0) return false;
    b = s.b;
    req = s.req;
    const long long base = U::before(*w, req, req.kb0);
    int lo = req.kb0, hi = req.kb1;  // H_kv * units before lo <= off < H_kv * units before hi
    while (hi - lo > 1) {
      const int mid = lo + ((hi - lo) >> 1);
      if (w->p.H_kv * (U::before(*w, req, mid) - base) <= s.off) lo = mid;
      else hi = mid;
    }
    kb = lo;
    low = U::m0(*w, req, kb);
    const long long off = s.off - w->p.H_kv * (U::before(*w, req, lo) - base);
    const int each = req.M - low + U::kRun;
    h = (int)(off / each);
    const int at = (int)(off - (long long)h * each);
    m = low + max(0, at - U::kRun);
    skip = max(0, U::kRun - at);
    whole = h == 0 && m == low;
    if (left <= skip) left = 0;  // its units end before the run's first tile
    return left > 0;
  }
  __device__ bool done() const { return left <= 0; }
  // tiles of this head and key block that follow each other here, this one first; walked in one step
  __device__ int run() const { return (int)min(left - skip, (long long)(req.M - m)); }
  // whether the run is the block's last with its key block
  __device__ bool keys_end(int run) const { return left - skip - run <= U::kRun || (h + 1 == w->p.H_kv && m + run == req.M); }
  // the key block's units behind the block's
  __device__ long long rest(int run) const {
    const long long behind = (long long)(w->p.H_kv - 1 - h) * (req.M - low + U::kRun) + req.M - m - run;
    return behind > 0 ? max(0ll, behind - (left - skip - run)) : 0;
  }
  __device__ void next(int run) {
    left -= skip + run;
    skip = 0;
    if (left <= 0) return;
    m += run;
    if (m < req.M) return;
    skip = U::kRun;
    m = low;
    if (++h == w->p.H_kv) {
      h = 0;
      whole = true;
      if (++kb == req.kb1) {
        do {
          req = U::request(*w, ++b);
        } while (req.kb0 == req.kb1);
        kb = req.kb0;
      }
      low = m = U::m0(*w, req, kb);
    }
    if (left <= skip) left = 0;
  }
  // rows of tile m: the first token, the first of its heads, and the columns that are rows of the request
  __device__ int token(int m) const { return (w->parts == 1 ? m : (int)quotient(m, w->by_parts)) * w->tokens; }
  __device__ int head(int m) const { return w->parts == 1 ? 0 : (m - (int)quotient(m, w->by_parts) * w->parts) * w->heads; }
  __device__ int columns(int m) const {
    return w->parts == 1 ? min(w->tokens, req.n - token(m)) * w->heads : min(w->heads, w->p.G - head(m));
  }
};

// Token j's slot, or -1: beyond the request, or on a page outside the pool.
__device__ __forceinline__ int weight_slot(const WeightParams& w, int b, int len, int j) {
  if (j >= len) return -1;
  const int i = (int)quotient(j, w.p.by_page), page = w.p.table[(size_t)b * w.p.table_stride + i];
  if ((unsigned)page >= (unsigned)w.p.n_pages) {
    if (w.p.status) atomicOr(w.p.status, GDN_STATUS_BAD_PAGE);
    return -1;
  }
  return page * w.p.page_size + j - i * w.p.page_size;
}
__device__ __forceinline__ bool weight_new(const WeightParams& w, const WeightRequest& r, int j) { return w.fresh && j >= r.ctx; }

// The place of a key's weight: kNewSlot on top of slots of tokens that start anew, -1 for none.
constexpr uint32_t kNewSlot = 1u << 31;
constexpr int kNoSlot = -1;
__device__ __forceinline__ int weight_place(const WeightParams& w, const WeightRequest& r, int b, int j) {
  const int slot = j >= r.first ? weight_slot(w, b, r.ctx + r.n, j) : kNoSlot;  // below 2^31 - 1: a pool has fewer slots
  return slot != kNoSlot && weight_new(w, r, j) ? (int)(slot | kNewSlot) : slot;
}
__device__ __forceinline__ void add_weight(const WeightParams& w, int place, float old, float got) {
  if (place == kNoSlot) return;
  w.weight[place & ~kNewSlot] = place < 0 ? got : fmaf(w.keep, old, got);
}
__device__ __forceinline__ float old_weight(const WeightParams& w, int place) { return place >= 0 ? w.weight[place] : 0.f; }

// Joins the partials of the key block that block blockIdx.x begins and does not end, and notes the step's own tokens' ages.
template <int kKeys>
__global__ void __launch_bounds__(kKeys) weight_join_kernel(const WeightParams w) {
  pdl_wait();
  pdl_trigger();
  const int followers = w.notes[blockIdx.x], place = w.slots[blockIdx.x * kKeys + threadIdx.x];
  float got = w.partials[(size_t)(2 * blockIdx.x + 1) * kKeys + threadIdx.x];
  if (followers > 0) {
    const float old = old_weight(w, place);
    for (int i = 1; i <= followers; ++i) got += w.partials[(size_t)(2 * (blockIdx.x + i)) * kKeys + threadIdx.x];
    add_weight(w, place, old, got);
  }
  if (w.fresh && w.born) {
    // blocks b, b + B, ... share request b's tokens
    const int shares = max(1, (int)gridDim.x / w.p.B);
    for (int b = blockIdx.x % w.p.B, share = blockIdx.x / w.p.B; b < w.p.B && share < shares; b += gridDim.x) {
      const Request r = request(w.p, b);
      const int position = r.n > 0 && w.position ? w.position[b] : r.ctx;
      for (long long t = share * kKeys + threadIdx.x; t < r.n; t += shares * kKeys) {
        const int slot = weight_slot(w, b, r.ctx + r.n, r.ctx + (int)t);
        if (slot >= 0) w.born[slot] = position + (int)t;
      }
    }
  }
}

// work: notes, places and partials of every block
inline size_t weight_work(int blocks, int keys) { return (size_t)blocks * (sizeof(int) + keys * (sizeof(int) + 2 * sizeof(float))); }
inline void set_weight_work(WeightParams& w, int blocks, int keys, void* work) {
  w.p.n_blocks = blocks;
  w.notes = static_cast<int*>(work);
  w.slots = w.notes + blocks;
  w.partials = reinterpret_cast<float*>(w.slots + (size_t)blocks * keys);
}
size_t weight_tc_work();
int run_weight_tc(WeightParams& w, void* work, cudaStream_t st);

// one tile's rows: as many tokens as fit `most` rows, but no more than a padded request has
inline void set_weight_tiles(WeightParams& w, int most) {
  w.heads = w.p.G < most ? w.p.G : most;
  w.parts = (w.p.G + w.heads - 1) / w.heads;
  w.tokens = w.parts > 1 ? 1 : most / w.heads;
  if (w.p.R > 0 && w.tokens > w.p.R) w.tokens = w.p.R;
  w.by_heads = make_div((uint32_t)w.heads);
  w.by_parts = make_div((uint32_t)w.parts);
}

template <int kKeys>
int launch_weight_join(const WeightParams& w, cudaStream_t st) {
  return launch(weight_join_kernel<kKeys>, dim3(w.p.n_blocks), dim3(kKeys), 0, st, w);
}

}  // namespace gdnattn
