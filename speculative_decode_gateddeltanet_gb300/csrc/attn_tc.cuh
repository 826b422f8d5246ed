// Paged attention in bf16 on the 5th-generation tensor cores: the kernel, for gdn_paged_attention and gdn_shared_attention.
//
// One block per SM walks its share of (tile of 128 rows, key block) units.  A
// tile's rows are the query heads of one kv head over its tokens, so K and V
// are read once for the whole group.  Per key block j:
//   S = Q K^T       tcgen05.mma, Q and K from shared memory, S (32-bit) in TMEM
//   P = 2^(s - m)   one thread per row: running maximum m, running sum, P to
//                   TMEM as bf16 over S's columns
//   O += P V        tcgen05.mma, P from TMEM, V from shared memory, O in TMEM
// Two streams (d <= 128).  A thread's 128 exponentials and what goes with them
// take longer than the two products, so two warpgroups halve a block's keys: each
// has its own O in TMEM and its own running maximum and sum, and the two are
// joined when the tile is written out; no word passes between them before that.
// Where O fills TMEM (d = 256) blocks have 64 keys and one warpgroup.  S has two
// buffers: the tensor cores form the next S while the softmax works on this one.
//
// Roles (512 threads): warps 0-3 and 4-7 softmax, warps 8-11 stage Q and write
// the tiles out (a TMEM lane is read by the warps of its quarter only), warp 12
// issues the first product's MMAs, warp 15 the second's (one thread for both would
// leave the tensor cores idle at each of its waits: 8192 tokens in 612 us, not 540), warps 13 and 14 the TMA copies
// of K and of V.
//
// Few rows.  A tile with few rows leaves softmax warps without one; those only keep
// step.  The MMA's 128 rows are paid for anyway.  (Staging few rows twice or four
// times, so that all warps share their exponentials, cost more in the join: 16
// requests of 4 tokens at d = 256 took 40.0 us, without 35.7.  Only d = 64, where a
// block's K and V arrive in less time than a warp needs for its rows, lost: 32
// tokens over 16000 took 99 us and take 109.)
//
// A page is copied in boxes of 64 columns by a power of two of tokens that
// divides the page, straight into the 128-byte-swizzled layout the MMA reads;
// pools of any strides are the tensor map's affair.  V is used as it lies (its
// columns are the MMA's N), so nothing is transposed.
//
// The running maximum is raised only when it would grow by more than 2^8:
// until then P stays below 2^8 and its sum is exact enough in 32 bits, and O
// (in TMEM) need not be rescaled.  P is rounded to bf16 for the second product
// (2^-9 of each weight); sums stay in 32 bits.
//
// Every wait is bounded by time; when one runs out the block flags it, sets
// GDN_STATUS_TIMEOUT, waits (bounded) for its own copies and products in
// flight, frees its TMEM and ends.
//
// Measured.  Prefill is bound by the chain of a block (scores, weights, products): a
// 128-key unit takes 0.86 us, where its MMAs alone take 0.53 and its softmax alone 0.40,
// so the two hardly overlap (8192 tokens at d = 128, 32 heads: 1.28 PFLOP/s, 0.69 of
// cuBLAS' bf16 rate; d = 256 1.19, d = 64 0.76).  Decode is bound by HBM behind a start of some 4 us
// (lengths, pages, the first copies) and an end of some 7 (tiles out, the join):
// 256 ragged requests of 2 to 9 tokens 167 to 170 us (6.0 TB/s, 0.88 of a copy's rate),
// one token over 65537 51 us (5.3 TB/s), 16 requests of 4 tokens over 1000 to 8000 at
// d = 256 35.1 us (4.1 TB/s).
#pragma once
#include <limits>
#include <type_traits>

#include "attn_tc.h"
#include "tc_ptx.cuh"

namespace gdnattn {

constexpr int kTcThreads = 512;
constexpr int kTcBlocks = 152;  // one block per SM of a GB300
constexpr int kTcMinUnits = 2;  // a block's least share: 4 tokens over 4000 take 16.0 us, with 4 16.8, with 1 15.9

template <int kD>
struct Shape {
  static constexpr int kKeys = kD == 256 ? 64 : 128;
  static constexpr int kChunks = kD / 64;                 // 128-byte column chunks of a row
  static constexpr int kQBytes = kTcRows * kD * 2;
  static constexpr int kTileBytes = kKeys * kD * 2;       // a K or V tile
  static constexpr int kK = kD == 64 ? 6 : kD == 128 ? 3 : 2;  // K tiles in flight
  static constexpr int kV = kD == 64 ? 5 : 2;
  static constexpr int kStreams = kD == 256 ? 1 : 2;      // TMEM: two S buffers and an O for each stream, of 512 columns
  static constexpr int kSmem = 1024 + kQBytes + (kK + kV) * kTileBytes;
};
static_assert(Shape<128>::kSmem <= 230 * 1024 && Shape<256>::kSmem <= 230 * 1024 && Shape<64>::kSmem <= 230 * 1024);

// a row's running softmax
struct RowState {
  float top, sum;
};

// One key block for this thread's row and its stream's kC columns: s_at is S in
// TMEM (this warp's lanes), edge the last column the row sees.  rescale(shrink)
// multiplies the row's O; it is called for whole warps.
// kFront: the first `front` columns are not the line's own.
template <int kC, bool kFront, typename Rescale>
__device__ __forceinline__ bool softmax_block(RowState& st, uint32_t s_at, int front, int edge, float scale_log2, Rescale rescale) {
  constexpr int kPart = 32;  // columns of one TMEM load
  uint32_t x[kC / kPart][kPart];
#pragma unroll
  for (int c = 0; c < kC / kPart; ++c) tmem_load(x[c], s_at + c * kPart);
  tmem_wait_load();
#pragma unroll
  for (int c = 0; c < kC / kPart; ++c) tmem_loaded(x[c]);
  if (edge < kC - 1) {
#pragma unroll
    for (int c = 0; c < kC / kPart; ++c)
#pragma unroll
      for (int i = 0; i < kPart; ++i)
        if (c * kPart + i > edge) x[c][i] = 0xff800000u;
  }
  if (kFront && front > 0) {
#pragma unroll
    for (int c = 0; c < kC / kPart; ++c)
#pragma unroll
      for (int i = 0; i < kPart; ++i)
        if (c * kPart + i < front) x[c][i] = 0xff800000u;
  }
  float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int c = 0; c < kC / kPart; ++c)
#pragma unroll
    for (int i = 0; i < kPart; ++i) m4[i & 3] = fmaxf(m4[i & 3], __uint_as_float(x[c][i]));
  const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * scale_log2;
  const bool raise = mx > st.top + 8.f;  // also the first time: top is -inf
  if (__any_sync(kFull, raise)) {
    const float shrink = raise ? ex2(st.top - mx) : 1.f;
    st.sum *= shrink;
    if (raise) st.top = mx;
    if (!rescale(shrink)) return false;
  }
  const float sub = st.top == -INFINITY ? 0.f : st.top;
  const uint64_t scale2 = pair(scale_log2, scale_log2), sub2 = pair(-sub, -sub);
  uint64_t s2[2] = {0, 0};
  constexpr int kW = 16;  // words of one TMEM store
#pragma unroll
  for (int c = 0; c < kC / 2; c += kW) {
    uint32_t pk[kW];
#pragma unroll
    for (int i = 0; i < kW; ++i) {
      const int j = 2 * (c + i);
      const float* const xs = reinterpret_cast<const float*>(x[j / kPart]) + j % kPart;
      const float2 y = halves(fma2(pair(xs[0], xs[1]), scale2, sub2)), e = {ex2(y.x), ex2(y.y)};
      s2[i & 1] = add2(s2[i & 1], pair(e.x, e.y));
      pk[i] = pack_bf16(e.x, e.y);
    }
    tmem_store(s_at + c, pk);  // over columns that were read
  }
  const float2 total = halves(add2(s2[0], s2[1]));
  st.sum += total.x + total.y;
  tmem_wait_store();
  return true;
}

#ifdef GDN_TEST_HOOKS
// Test builds only: the block whose first K copy is declared on its barrier but never issued (-1: none).
__device__ int g_test_drop_block = -1;
#endif

struct TcParams {
  Params p;
  int box;          // tokens per TMA box: a power of two that divides the page and kKeys
  uint32_t q_flip;  // sign bits to flip in q: a negative scale is taken into q, exactly
};

// kShared: the lines of gdn_shared_attention in place of requests, a tile's first part left in `dense` for its rows' join
template <int kD, bool kShared>
__global__ void __launch_bounds__(kTcThreads, 1)
    tc_kernel(const TcParams t, const std::conditional_t<kShared, SharedParams, Nothing> sp, const __grid_constant__ CUtensorMap k_map,
              const __grid_constant__ CUtensorMap v_map) {
  using S = Shape<kD>;
  using W = Walk<kTcRows, S::kKeys, kShared>;
  constexpr int kKeys = S::kKeys, kChunks = S::kChunks;
  const Params& p = t.p;
  const uint32_t q_flip = t.q_flip;
  extern __shared__ __align__(16) uint8_t raw[];
  __shared__ __align__(8) uint64_t bars[2 * S::kK + 2 * S::kV + 15 + kShared];
  __shared__ long long scan[(kShared ? 3 : 1) * kTcThreads / 32];
  __shared__ StartOf<typename W::R> start;
  __shared__ int row_at[kShared ? 2 : 1][kShared ? kTcRows : 1];  // by tile: its rows' rows of q and o
  __shared__ uint32_t tmem_base;
  __shared__ int gave_up;
  __shared__ float2 stats[2][2][128];  // maxima and sums of a tile's rows, by tile and stream
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
  const uint32_t q_s = base, k_s = q_s + S::kQBytes, v_s = k_s + S::kK * S::kTileBytes;
  // A wait names a phase by its parity, so a barrier may be at most one phase ahead of any of its waiters, and each
  // waiter takes every phase in turn, or knows from another wait that the one before has passed; what may be signalled
  // twice before it is waited for has two barriers.  Waits are few on purpose: one costs some 50 ns even when it is over
  // (a third wait a block in the softmax cost 5 % of a prompt's time, separate ones for the streams' P another 3 %), and
  // polling instead of suspending 25 %.
  const uint32_t b0 = smem_addr(bars);
  auto k_full = [&](int i) { return b0 + 8 * i; };
  auto k_empty = [&](int i) { return b0 + 8 * (S::kK + i); };
  auto v_full = [&](int i) { return b0 + 8 * (2 * S::kK + i); };
  auto v_empty = [&](int i) { return b0 + 8 * (2 * S::kK + S::kV + i); };
  constexpr int kRest = 2 * S::kK + 2 * S::kV;
  auto s_full = [&](int i) { return b0 + 8 * (kRest + (i & 1)); };       // S of block i is in TMEM
  auto p_ready = [&](int i) { return b0 + 8 * (kRest + 2 + (i & 1)); };  // P of it is, of all streams
  auto pv_done = [&](int i) { return b0 + 8 * (kRest + 4 + (i & 1)); };  // O holds its products
  auto st_ready = [&](int g) { return b0 + 8 * (kRest + 6 + (g & 1)); };  // tile g's maxima and sums are in `stats`
  auto o_full = [&](int g) { return b0 + 8 * (kRest + 8 + (g & 1)); };   // tile g's O is whole
  auto o_free = [&](int g) { return b0 + 8 * (kRest + 10 + (g & 1)); };   // and has been written out
  const uint32_t q_full = b0 + 8 * (kRest + 12), q_empty = b0 + 8 * (kRest + 13), drained = b0 + 8 * (kRest + 14);
  const uint32_t row_ready = b0 + 8 * (kRest + 15);  // kShared: row_at holds a tile's rows
  if (tid == 0) {
    gave_up = 0;
    for (int i = 0; i < S::kK; ++i) {
      bar_init(k_full(i), 1);
      bar_init(k_empty(i), 1);
    }
    for (int i = 0; i < S::kV; ++i) {
      bar_init(v_full(i), 1);
      bar_init(v_empty(i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(s_full(i), 1);
      bar_init(p_ready(i), 4 * S::kStreams);
      bar_init(pv_done(i), 1);
      bar_init(st_ready(i), 4 * S::kStreams);
      bar_init(o_full(i), 1);
      bar_init(o_free(i), 4);
    }
    bar_init(q_full, 4);
    bar_init(q_empty, 1);
    bar_init(drained, 2);
    if (kShared) bar_init(row_ready, 4);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&tmem_base)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == 13 && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&k_map) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&v_map) : "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  pdl_trigger();
  const uint32_t tmem = tmem_base;
  Lines lines = {};
  if constexpr (kShared)
    lines = find_lines<kTcRows, kKeys, kTcThreads>(p, sp, kTcMinUnits, reinterpret_cast<int*>(raw + S::kSmem), scan, &start);
  else
    find_start<kTcRows, kKeys, kTcThreads>(p, kTcMinUnits, scan, &start);
  const auto s = start;
  constexpr uint32_t kOCol = 2 * kKeys;  // TMEM columns: two S buffers, then O
  constexpr int kCols = kKeys / S::kStreams;  // a stream's keys of a block
  W w;
  if constexpr (kShared) {
    w.lines = &lines;
    w.align = sp.key_align;
  }
  const bool any = begin(w, p, s);
  bool ok = true;
  int sent = 0;  // tiles whose copies this warp issued
  // whether the tile's rows have parts over a prefix and over their own keys
  auto joins = [](const W& t) {
    if constexpr (kShared) return t.req.prefix != 0;
    else return false;
  };
  auto rows_of = [&](const W& t) {
    return (int)min((long long)kTcRows, (long long)t.req.n * p.G - (long long)t.m * kTcRows);
  };

  if (warp >= 8 && warp < 12) {
    // ---- Q into the swizzled layout, and the tiles out of TMEM
    int4 note = {0, 0, 0, 0};
    if (any) {
      const int e_tid = tid - 256, quarter = warp - 8;
      const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
      constexpr int kUnits = kD / 8;  // 16-byte units of a row
      constexpr int kBatch = 8;       // units a thread has under way
      auto stage_q = [&](const W& t, int g) {
        const int rows = rows_of(t);
        if constexpr (kShared) {
          const int at = min(t.m * kTcRows + e_tid, t.req.n * p.G - 1);
          row_at[g & 1][e_tid] = lines.row_of(p, t.req, (int)quotient(at, p.by_G));
          warp_arrive(row_ready);
          if (!warp_wait(row_ready, g & 1, &gave_up)) return false;
        }
        for (int i0 = 0; i0 < rows * kUnits; i0 += kBatch * 128) {
          uint4 x[kBatch];
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            // past the tile's rows its last one again: no load hides behind a branch
            const int i = i0 + j * 128 + e_tid, r = min(i / kUnits, rows - 1), u = i % kUnits, at = t.m * kTcRows + r;
            const int token = (int)quotient(at, p.by_G), head = t.h * p.G + at - token * p.G;
            int q_row;
            if constexpr (kShared) q_row = row_at[g & 1][r];
            else q_row = t.req.row0 + token;
            x[j] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + (int64_t)q_row * p.q_row +
                                                        (int64_t)head * p.q_head + u * 8));
          }
          // the rows are on their way while the last tile's products with Q end
          if (i0 == 0 && g > 0 && !warp_wait(q_empty, (g - 1) & 1, &gave_up)) return false;
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            const int i = i0 + j * 128 + e_tid;
            if (i < rows * kUnits) {
              const int r = i / kUnits, u = i % kUnits;
              const uint32_t to = q_s + (u / 8) * (kTcRows * 128) + r * 128 + (((u & 7) ^ (r & 7)) << 4);
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(x[j].x ^ q_flip), "r"(x[j].y ^ q_flip),
                           "r"(x[j].z ^ q_flip), "r"(x[j].w ^ q_flip)
                           : "memory");
            }
          }
        }
        fence_async();
        warp_arrive(q_full);
        return true;
      };
      ok = stage_q(w, 0);
      for (int g = 0; ok && !w.done(); ++g) {
        W next = w;
        next.next();
        int o_row = 0;
        if constexpr (kShared) o_row = row_at[g & 1][e_tid];
        if (!next.done() && !(ok = stage_q(next, g + 1))) break;
        const int rows = rows_of(w), row = e_tid;
        const int at = min(w.m * kTcRows + row, w.req.n * p.G - 1);
        const int token = (int)quotient(at, p.by_G), head = w.h * p.G + at - token * p.G;
        const bool whole = w.kb0 == 0 && w.kb1 == w.blocks && !joins(w);
        const int slot = w.kb0 == 0 ? 1 : 0;
        float* const part = partial(p, blockIdx.x, slot, kTcRows);
        float* out = part + row * kD;  // this row's 32-bit columns
        float2* out_stats = reinterpret_cast<float2*>(part + kTcRows * kD) + row;
        bool first = false;  // of a row that takes part in a prefix
        if constexpr (kShared) {
          if (joins(w) && w.kb0 == 0) {
            const size_t place = place_of(p, sp, !w.req.flat(), lines.rank_of(w.req, token), w.h, head - w.h * p.G);
            first = true;
            out = sp.dense + place * kD;
            out_stats = reinterpret_cast<float2*>(sp.entries + place);
          }
        } else {
          o_row = w.req.row0 + token;
        }
        if (!whole && !first && slot == 1) note = note_of(w, s);
        __nv_bfloat16* const dst = static_cast<__nv_bfloat16*>(p.o) + (int64_t)o_row * p.o_row + (int64_t)head * p.o_head;
        ok = warp_wait(st_ready(g), (g >> 1) & 1, &gave_up) && warp_wait(o_full(g), (g >> 1) & 1, &gave_up);
        if (!ok) break;
        tc_fence_after();
        // the second stream has no O where the tile's only block ends before its keys
        const int n_parts = S::kStreams == 1 || (w.kb1 - w.kb0 == 1 && w.req.len() - w.kb0 * kKeys <= kCols) ? 1 : 2;
        if (quarter * 32 < rows) {
          const float2 st0 = stats[g & 1][0][row], st1 = n_parts == 2 ? stats[g & 1][1][row] : make_float2(-INFINITY, 0.f);
          const float top = fmaxf(st0.x, st1.x), sub = top == -INFINITY ? 0.f : top;
          float share0 = ex2(st0.x - sub), share1 = ex2(st1.x - sub);  // 2^(own maximum - common maximum)
          const float sum = st0.y * share0 + st1.y * share1;
          if (!whole && row < rows) *out_stats = make_float2(top, sum);
          if constexpr (kShared) {
            if (row < rows && first) reinterpret_cast<int2*>(out_stats)[1] = make_int2(blockIdx.x, entry_word(followers_of(w, s), row));
            if (row < rows && whole && sp.lse) sp.lse[(int64_t)o_row * sp.lse_row + head] = (top + log2f(sum)) * kLn2;
          }
          if (whole) {
            share0 /= sum;
            share1 /= sum;
          }
          // 32 columns of this lane's row, the streams added up
          auto columns = [&](float (&v)[32], int c) {
            uint32_t o0[32], o1[32];
            tmem_load(o0, lanes + kOCol + c * 32);
            if (n_parts == 2) tmem_load(o1, lanes + kOCol + kD + c * 32);
            tmem_wait_load();
            tmem_loaded(o0);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(o0[i]) * share0;
            if (n_parts == 2) {
              tmem_loaded(o1);
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = fmaf(__uint_as_float(o1[i]), share1, v[i]);
            }
          };
#pragma unroll 1
          for (int c = 0; c < kD / 32; ++c) {
            float v[32];
            columns(v, c);
            if (row < rows) {
              if (whole) {
                uint32_t pk[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) pk[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  reinterpret_cast<uint4*>(dst + c * 32)[i] = make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
              } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  reinterpret_cast<float4*>(out + c * 32)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
              }
            }
          }
        }
        tc_fence_before();
        warp_arrive(o_free(g));
        w = next;
      }
    }
    if (tid == 256) p.notes[blockIdx.x] = note;
  } else if (any && warp < 4 * S::kStreams) {
    // ---- softmax: one thread per row, the stream's keys
    const int stream = warp >> 2, quarter = warp & 3, s_tid = tid & 127;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    int it = 0, g = 0;
    for (; ok && !w.done(); w.next(), ++g) {
      const int rows = rows_of(w), row = s_tid;
      const bool active = quarter * 32 < rows;  // a warp with no row only keeps step
      const int last = row < rows ? w.req.last((int)quotient(w.m * kTcRows + row, p.by_G)) : -1;
      RowState st = {-INFINITY, 0.f};
      for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
        if (!(ok = warp_wait(s_full(it), (it >> 1) & 1, &gave_up))) break;
        if (active) {
          tc_fence_after();
          auto rescale = [&](float shrink) {
            if (kb == w.kb0) return true;
            // this S was formed behind block it - 2's products, the one wait that is not taken
            if (!warp_wait(pv_done(it - 1), ((it - 1) >> 1) & 1, &gave_up)) return false;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < kD / 32; ++c) {
              uint32_t o[32];
              tmem_load(o, lanes + kOCol + stream * kD + c * 32);
              tmem_wait_load();
              tmem_loaded(o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * shrink);
              tmem_store(lanes + kOCol + stream * kD + c * 32, o);
            }
            tmem_wait_store();
            return true;
          };
          const int edge = last - kb * kKeys - stream * kCols;
          const uint32_t s_at = lanes + (it & 1) * kKeys + stream * kCols;
          int front = 0;
          if constexpr (kShared) front = kb == 0 ? w.req.front - stream * kCols : 0;
          ok = softmax_block<kCols, kShared>(st, s_at, front, edge, p.scale_log2, rescale);
          if (!ok) break;
          tc_fence_before();
        }
        const int valid = w.req.len() - kb * kKeys;
        if (valid < kKeys && valid % 16 != 0 && valid / kCols == stream) {
          // The V rows between the request's last token and the last 16 that the MMA reads: their weight is 0, but 0
          // times what a page holds there may be NaN.
          const int vs = it % S::kV;
          if (!(ok = warp_wait(v_full(vs), (it / S::kV) & 1, &gave_up))) break;
          for (int i = s_tid; i < (16 - valid % 16) * (kD / 8); i += 128) {
            const int r = valid + i / (kD / 8), u = i % (kD / 8);
            const uint32_t to = v_s + vs * S::kTileBytes + (u / 8) * (kKeys * 128) + r * 128 + ((u & 7) << 4);
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(to), "r"(0) : "memory");
          }
          fence_async();
        }
        warp_arrive(p_ready(it));
      }
      if (ok && g >= 2) ok = warp_wait(o_free(g), ((g >> 1) - 1) & 1, &gave_up);  // tile g - 2 is done with its place in stats
      if (!ok) break;
      stats[g & 1][stream][s_tid] = make_float2(st.top, st.sum);
      warp_arrive(st_ready(g));
    }
  } else if (any && warp == 12) {
    // ---- S = Q K^T, issued by one thread
    if (lane == 0) {
      constexpr uint32_t kQk = instruction(kKeys, false);
      const uint32_t q_lo = operand_lo(q_s, 16), k_lo0 = operand_lo(k_s, 16);
      uint32_t stage = 0, k_phase = 0, buf = 0, s_phase = 1, q_phase = 0;  // s_phase: of pv_done; the first round finds S free
      for (; ok && !w.done(); w.next()) {
        if (!(ok = bar_wait(q_full, q_phase, &gave_up))) break;
        q_phase ^= 1;
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          // the products of the buffer's last P are done
          ok = bar_wait(k_full(0) + 8 * stage, k_phase, &gave_up) && bar_wait(pv_done(0) + 8 * buf, s_phase, &gave_up);
          if (!ok) break;
          tc_fence_after();
          const uint32_t k_lo = k_lo0 + stage * (S::kTileBytes / 16), s_at = tmem + buf * kKeys;
#pragma unroll
          for (int k = 0; k < kD / 16; ++k)
            mma_ss(s_at, q_lo + (k / 4) * (kTcRows * 8) + (k % 4) * 2, k_lo + (k / 4) * (kKeys * 8) + (k % 4) * 2, kOperandHi, kQk, k > 0);
          tc_commit(s_full(0) + 8 * buf);
          tc_commit(k_empty(0) + 8 * stage);
          if (kb == w.kb1 - 1) tc_commit(q_empty);
          s_phase ^= buf;
          buf ^= 1;
          if (++stage == S::kK) {
            stage = 0;
            k_phase ^= 1;
          }
        }
      }
    }
    __syncwarp();
  } else if (any && warp == 15) {
    // ---- O += P V, issued by one thread
    if (lane == 0) {
      constexpr uint32_t kPv = instruction(kD, true);
      const uint32_t v_lo0 = operand_lo(v_s, kKeys * 128);
      uint32_t stage = 0, v_phase = 0, buf = 0, p_phase = 0, o_phase = 0;  // o_phase: of o_free's two barriers in turn
      int g = 0;
      for (; ok && !w.done(); w.next(), ++g) {
        const int len = w.req.len();
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          const uint32_t fresh = kb > w.kb0;  // 0: the tile's first block overwrites O
          const int valid = len - kb * kKeys;
          const uint32_t v_lo = v_lo0 + stage * (S::kTileBytes / 16), p_at = tmem + buf * kKeys;
          ok = bar_wait(v_full(0) + 8 * stage, v_phase, &gave_up);
          if (!fresh && g > 0) {  // the last tile has been written out
            ok = ok && bar_wait(o_free(g - 1), o_phase >> 1, &gave_up);
            o_phase = (o_phase + 1) & 3;
          }
          ok = ok && bar_wait(p_ready(0) + 8 * buf, p_phase, &gave_up);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int x = 0; x < S::kStreams; ++x) {
            const uint32_t o_at = tmem + kOCol + x * kD, px_at = p_at + x * kCols, v_at = v_lo + x * (kCols * 8);
            if (valid >= (x + 1) * kCols) {
#pragma unroll
              for (int k = 0; k < kCols / 16; ++k) mma_ts(o_at, px_at + k * 8, v_at + k * 128, kOperandHi, kPv, k > 0 ? 1u : fresh);
            } else {
              const int steps = (valid - x * kCols + 15) >> 4;  // no V row behind the last 16 with a token
              for (int k = 0; k < steps; ++k) mma_ts(o_at, px_at + k * 8, v_at + k * 128, kOperandHi, kPv, k > 0 ? 1u : fresh);
            }
          }
          if (!ok) break;
          tc_commit(pv_done(0) + 8 * buf);
          tc_commit(v_empty(0) + 8 * stage);
          if (kb == w.kb1 - 1) tc_commit(o_full(g));
          p_phase ^= buf;
          buf ^= 1;
          if (++stage == S::kV) {
            stage = 0;
            v_phase ^= 1;
          }
        }
      }
    }
    __syncwarp();
  } else if (any && (warp == 13 || warp == 14)) {
    // ---- K (warp 13) and V (warp 14) tiles by TMA: lane (box, chunk) copies its box of 64 columns
    const bool is_v = warp == 14;
    const int stages = is_v ? S::kV : S::kK;
    const uint32_t tiles = is_v ? v_s : k_s, full = is_v ? v_full(0) : k_full(0), empty = is_v ? v_empty(0) : k_empty(0);
    const CUtensorMap* const map = is_v ? &v_map : &k_map;
    const int n_box = kKeys / t.box, box = lane / kChunks, chunk = lane % kChunks;
    const uint32_t at = (uint32_t)chunk * (kKeys * 128) + (uint32_t)box * t.box * 128;
    int stage = 0;
    uint32_t phase = 1;  // of `empty`: the first round finds the stages free
    for (; ok && !w.done(); w.next()) {
      const int len = w.req.len(), first_key = w.first_key();
      const int32_t* const row = p.table + (size_t)w.table_row() * p.table_stride;
      struct Box {
        int page, token;
      };
      auto find_page = [&](int kb) -> Box {
        const int j = kb * kKeys + box * t.box;
        if (kb >= w.kb1 || box >= n_box || j >= len) return {0, 0};
        const int key = first_key + j, i = (int)quotient(key, p.by_page);
        return {row[i], key - i * p.page_size};
      };
      Box next[2] = {find_page(w.kb0), find_page(w.kb0 + 1)};  // two blocks ahead: a table entry is a round trip to L2
      for (int kb = w.kb0; kb < w.kb1; ++kb) {
        const int live = min(n_box, (len - kb * kKeys + t.box - 1) / t.box);
        int my_page = next[0].page;
        const int my_token = next[0].token;
        next[0] = next[1];
        next[1] = find_page(kb + 2);
        if (!(ok = warp_wait(empty + 8 * stage, phase, &gave_up))) break;
        if (lane == 0) bar_expect(full + 8 * stage, (uint32_t)live * t.box * kD * 2);
        __syncwarp();
        if ((unsigned)my_page >= (unsigned)p.n_pages) {
          my_page = p.n_pages;  // outside the map: zeros
          if (p.status) atomicOr(p.status, GDN_STATUS_BAD_PAGE);
        }
#ifdef GDN_TEST_HOOKS
        const bool issue = is_v || sent > 0 || (int)blockIdx.x != g_test_drop_block;
#else
        constexpr bool issue = true;
#endif
        if (issue && box < live) tma_box(map, tiles + stage * S::kTileBytes + at, full + 8 * stage, chunk * 64, my_token, w.h, my_page);
        ++sent;
        if (++stage == stages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
  }
  __syncthreads();
  if (gave_up) {
    // products and copies that may still be in flight, with a bound again
    const unsigned long long end = now_ns() + kWaitNs;
    if (tid == 12 * 32 || tid == 15 * 32) {
      tc_commit(drained);
      while (!bar_try(drained, 0) && now_ns() < end) {
      }
    }
    if (lane == 0 && (warp == 13 || warp == 14)) {
      const int stages = warp == 13 ? S::kK : S::kV;
      for (int i = max(0, sent - stages); i < sent; ++i)
        while (!bar_try((warp == 13 ? k_full(0) : v_full(0)) + 8 * (i % stages), (i / stages) & 1) && now_ns() < end) {
        }
    }
    if (tid == 0 && p.status) atomicOr(p.status, GDN_STATUS_TIMEOUT);
    __syncthreads();
  }
  if (warp == 12) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// Launches the attention and the join of its parts.
template <int kD, bool kShared>
int run(TcParams& t, std::conditional_t<kShared, SharedParams, Nothing> sp, cudaStream_t st) {
  using S = Shape<kD>;
  size_t smem = S::kSmem;
  if constexpr (kShared) smem += sizeof(int) * lines_words(t.p.B, sp.n_groups);
  if (cudaFuncSetAttribute(tc_kernel<kD, kShared>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kShared ? S::kSmem + (int)sizeof(int) * kMaxLinesWords : S::kSmem) != cudaSuccess)
    return GDN_ERR_LAUNCH;
  t.box = 16;
  while (t.box * 2 <= S::kKeys && t.p.page_size % (t.box * 2) == 0) t.box *= 2;
  if constexpr (kShared) sp.key_align = t.box;
  CUtensorMap k_map, v_map;
  if (!make_map(&k_map, t.p, t.p.k, t.p.k_token, t.p.k_head, t.p.k_page, t.box) ||
      !make_map(&v_map, t.p, t.p.v, t.p.v_token, t.p.v_head, t.p.v_page, t.box))
    return GDN_ERR_LAUNCH;
  t.p.n_blocks = kTcBlocks;
  const int rc = launch(tc_kernel<kD, kShared>, dim3(kTcBlocks), dim3(kTcThreads), smem, st, t, sp, k_map, v_map);
  if (rc != GDN_OK) return rc;
  if constexpr (kShared) return launch_combine_shared<__nv_bfloat16, kD, kTcRows>(t.p, sp, st);
  else return launch(combine_kernel<__nv_bfloat16, kD, kTcRows>, dim3(kTcBlocks, 8), dim3(32 * kCombineWarps), 0, st, t.p);
}

template <bool kShared>
int run(const Params& p, const std::conditional_t<kShared, SharedParams, Nothing>& sp, cudaStream_t st) {
  TcParams t{p, 0, 0};
  if (t.p.scale_log2 < 0.f) {
    t.q_flip = 0x80008000u;
    t.p.scale_log2 = -t.p.scale_log2;
  }
  // a hidden score is -inf, and -inf * 0 would be NaN; the smallest number leaves no score as much as 1e-6
  if (t.p.scale_log2 == 0.f) t.p.scale_log2 = std::numeric_limits<float>::denorm_min();
  return p.d == 64 ? run<64, kShared>(t, sp, st) : p.d == 128 ? run<128, kShared>(t, sp, st) : run<256, kShared>(t, sp, st);
}

}  // namespace gdnattn
