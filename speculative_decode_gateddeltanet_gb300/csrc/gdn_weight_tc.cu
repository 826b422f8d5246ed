// Attention weights in bf16 on the 5th-generation tensor cores.
//
// One block per SM walks its units (weight_common.cuh).  For each:
//   S = K Q^T   tcgen05.mma: 128 keys by a tile's rows, K and Q by TMA into the MMA's layout, S (32-bit) in TMEM
//   got += sum over S's columns of 2^(log2(e) (scale s - lse))
// Keys are S's lanes: a thread owns a key and adds up its own columns, so no number crosses a thread, and a key's sum
// over rows and heads stays in a register until its block of keys is done.  A tile's sum, a head's and the heads' are
// separate sums in 32 bits: one chain over a prompt's 10^5 rows and heads would lose 4e-6.
//
// Roles (512 threads): three groups of four warps take the tiles out of TMEM in turn (four S buffers), warp 12 issues the
// products, warp 13 copies K, warp 14 Q, warp 15 the rows' lse (one warp for both took 1500 clocks a tile, more than its
// sums).  K of a (key block, head) is loaded once and met by all its tiles; a single step's few rows are one tile, and then K
// streams through.
//
// Measured.  Prompts: 8192 tokens at d = 128, 32 heads 258 us (1.07 PFLOP/s), at d = 64 220, at d = 256 (64 rows a tile) 338;
// 1500 to 4096 tokens of two requests 79.  A tile of 128 x 128 takes 1250 clocks, where its products and its exponentials
// take 512 each: bound by instructions (issue 62 %, exponentials 51 % of their rate).  Steps: 16 requests of 4 tokens over 1000
// to 8000 at d = 256 17.9 us, of which 3 are HBM's wait for the first K and 9 the stream at HBM's rate; one token over 65537
// at d = 128 40, where a unit takes 0.95 us and its 32 KB of K 0.72: without K, Q and sums it would still take 34, the roles'
// own steps between their waits.
//
// K's pages are copied whole, by one instruction (an instruction for each chunk of 16 tokens takes the issuing lane some 80 to
// 150 clocks; 32 of them for 64 KB took longer than HBM).
//
// Rows past the request's, and keys past its last token, may hold anything: a column or a lane is one row or key, and
// theirs are not counted.
#include <cuda.h>

#include <limits>

#include "tc_ptx.cuh"
#include "weight_common.cuh"

namespace gdnattn {

constexpr int kGroups = 3, kWeightThreads = 128 * kGroups + 128, kWeightBlocks = 152, kWeightKeys = 128;

template <int kD>
struct WeightShape {
  static constexpr int kRows = kD == 256 ? 64 : 128;  // a tile's most rows: S's columns
  static constexpr int kChunks = kD / 64;
  static constexpr int kKBytes = kWeightKeys * kD * 2, kQBytes = kRows * kD * 2;
  // Stages: of K at least so many, the rest is shared out by the size of a tile (run).
  static constexpr int kLeastK = kD == 64 ? 6 : kD == 128 ? 3 : 2, kMostK = 8, kMostQ = 8;
  static constexpr int kBytes = 216 * 1024;  // of both
  static constexpr int kSmem = 1024 + kBytes;
};
static_assert(WeightShape<64>::kLeastK * WeightShape<64>::kKBytes + 2 * WeightShape<64>::kQBytes <= WeightShape<64>::kBytes);
static_assert(WeightShape<128>::kLeastK * WeightShape<128>::kKBytes + 2 * WeightShape<128>::kQBytes <= WeightShape<128>::kBytes);
static_assert(WeightShape<256>::kLeastK * WeightShape<256>::kKBytes + 2 * WeightShape<256>::kQBytes <= WeightShape<256>::kBytes);

__device__ __forceinline__ void tma_rows(const CUtensorMap* map, uint32_t dst, uint32_t bar, int col, int head, int row) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(col), "r"(head), "r"(row), "r"(bar)
      : "memory");
}
#ifdef GDN_TEST_HOOKS
// Test builds only: the block whose first K copy is declared on its barrier but never issued (-1: none).
__device__ int g_test_drop_block = -1;
#endif

struct WeightTcParams {
  WeightParams w;
  int box;    // tokens per TMA box of K
  int width;  // columns of a product: a tile's rows up to a multiple of 16
  int n_k, n_q;  // stages
  PageMap k_pages;
};

template <int kD>
__global__ void __launch_bounds__(kWeightThreads, 1)
    weight_tc_kernel(const WeightTcParams t, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap q_map) {
  using S = WeightShape<kD>;
  constexpr int kKeys = kWeightKeys, kChunks = S::kChunks, kS = 4, kL = 8;
  const WeightParams& w = t.w;
  const Params& p = w.p;
  extern __shared__ __align__(16) uint8_t raw[];
  __shared__ __align__(8) uint64_t bars[2 * S::kMostK + 2 * S::kMostQ + kS + 5 + 3 * kL];
  __shared__ long long scan[kWeightThreads / 32];
  __shared__ WeightStart start;
  __shared__ uint32_t tmem_base;
  __shared__ int gave_up;
  __shared__ __align__(16) float lse_s[kL][S::kRows];
  __shared__ float cross[2][kGroups - 1][kKeys];  // the other groups' sums, by key block
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = (smem_addr(raw) + 1023) & ~1023u, k_s = base, q_s = k_s + t.n_k * S::kKBytes, q_bytes = t.width * kD * 2;
  const uint32_t b0 = smem_addr(bars);
  auto k_full = [&](int i) { return b0 + 8 * i; };
  auto k_empty = [&](int i) { return b0 + 8 * (S::kMostK + i); };
  auto q_full = [&](int i) { return b0 + 8 * (2 * S::kMostK + i); };
  auto q_empty = [&](int i) { return b0 + 8 * (2 * S::kMostK + S::kMostQ + i); };
  constexpr int kRest = 2 * S::kMostK + 2 * S::kMostQ;
  auto s_empty = [&](int i) { return b0 + 8 * (kRest + i); };
  auto c_full = [&](int i) { return b0 + 8 * (kRest + kS + i); };       // cross holds a key block's sums
  auto c_empty = [&](int i) { return b0 + 8 * (kRest + kS + 2 + i); };  // and they have been read
  const uint32_t drained = b0 + 8 * (kRest + kS + 4);
  // lse has a ring of its own: it is read until a tile's sums are done, some 2000 clocks after Q is free again
  auto l_empty = [&](int i) { return b0 + 8 * (kRest + kS + 5 + i); };
  // A wait names a phase by its parity, so a waiter must know that the phase before has passed.  A group waits for every third
  // tile: that tile i - 3 is there, by its own wait, says that tile i - kL is, as products and lse come in order.
  auto s_full = [&](int i) { return b0 + 8 * (kRest + kS + 5 + kL + i % kL); };
  auto l_full = [&](int i) { return b0 + 8 * (kRest + kS + 5 + 2 * kL + i % kL); };
  if (tid == 0) {
    gave_up = 0;
    for (int i = 0; i < t.n_k; ++i) {
      bar_init(k_full(i), 1);
      bar_init(k_empty(i), 1);
    }
    for (int i = 0; i < t.n_q; ++i) {
      bar_init(q_full(i), 1);
      bar_init(q_empty(i), 1);
    }
    for (int i = 0; i < kL; ++i) {
      bar_init(s_full(i), 1);
      bar_init(l_full(i), 1);
      bar_init(l_empty(i), 4);
    }
    for (int i = 0; i < kS; ++i) bar_init(s_empty(i), 4);
    for (int i = 0; i < 2; ++i) {
      bar_init(c_full(i), 4 * (kGroups - 1));
      bar_init(c_empty(i), 4);
    }
    bar_init(drained, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&tmem_base)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == 13 && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&k_map) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&q_map) : "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  pdl_trigger();
  const uint32_t tmem = tmem_base;
  find_weight_start<kKeys, kWeightThreads>(w, scan, &start);
  WeightWalk<kKeys> x;
  const bool any = x.begin(w, start);
  bool ok = true;
  int sent = 0;  // copies this warp issued
  // a ring's stage and the parity of its round; one more step
  struct Ring {
    int stage, round, size;
    __device__ void next() {
      if (++stage == size) {
        stage = 0;
        ++round;
      }
    }
  };
  Ring q_ring = {0, 0, t.n_q}, k_ring = {0, 0, t.n_k};

  if (any && warp < 4 * kGroups) {
    // ---- S out of TMEM, the groups in turn; the first also writes the weights
    const int group = warp >> 2, quarter = warp & 3, key = tid & 127;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint64_t scale2 = pair(p.scale_log2, p.scale_log2);
    float in_keys = 0.f, in_head = 0.f;  // sums over the key block's heads before this one, and over this head's tiles
    int place = 0;  // of this thread's key's weight, and what it holds
    float old = 0.f;
    bool known = false;
    int note = 0;
    auto look_up = [&]() {
      place = weight_place(w, x.req, x.b, x.kb * kKeys + key);
      old = old_weight(w, place);
      known = true;
    };
    int done = 0, turn = 0, f = 0;  // tiles so far, whose turn it is, key blocks
    for (int run; !x.done(); x.next(run)) {
      run = x.run();
      int r = group - turn;  // the group's first tile of the run
      if (r < 0) r += kGroups;
      const int past0 = x.kb * kKeys + key - x.req.ctx;
      for (; r < run; r += kGroups) {
        const int i = done + r, m = x.m + r, buf = i % kS, stage = i % kL;
        if (!(ok = warp_wait(s_full(i), (i / kL) & 1, &gave_up) && warp_wait(l_full(i), (i / kL) & 1, &gave_up))) break;
        tc_fence_after();
        const int n_cols = x.columns(m), past = past0 - x.token(m);
        // a row's token t sees this key where t >= past; no key of the block is hidden where the last is not
        const int from = past - key + kKeys - 1 > 0 ? past * w.heads : 0;
        uint64_t sum2[2] = {0, 0};
        auto sum_up = [&](const uint32_t (&s)[32], int c) {
          auto term = [&](int k, float2 l) {  // columns c + k and the next
            const float* const v = reinterpret_cast<const float*>(s) + k;
            const float2 y = halves(fma2(pair(v[0], v[1]), scale2, pair(l.x, l.y)));
            return make_float2(ex2(y.x), ex2(y.y));
          };
          if (__all_sync(kFull, c >= from && c + 32 <= n_cols)) {
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
              const float4 l = *reinterpret_cast<const float4*>(&lse_s[stage][c + k]);
              const float2 e0 = term(k, make_float2(l.x, l.y)), e1 = term(k + 2, make_float2(l.z, l.w));
              sum2[0] = add2(sum2[0], pair(e0.x, e0.y));
              sum2[1] = add2(sum2[1], pair(e1.x, e1.y));
            }
          } else {
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
              const float4 l = *reinterpret_cast<const float4*>(&lse_s[stage][c + k]);
              float2 e0 = term(k, make_float2(l.x, l.y)), e1 = term(k + 2, make_float2(l.z, l.w));
              const int at = c + k;
              if (at < from || at >= n_cols) e0.x = 0.f;
              if (at + 1 < from || at + 1 >= n_cols) e0.y = 0.f;
              if (at + 2 < from || at + 2 >= n_cols) e1.x = 0.f;
              if (at + 3 < from || at + 3 >= n_cols) e1.y = 0.f;
              sum2[0] = add2(sum2[0], pair(e0.x, e0.y));
              sum2[1] = add2(sum2[1], pair(e1.x, e1.y));
            }
          }
        };
#pragma unroll 1
        for (int c = 0; c < n_cols; c += 32) {
          uint32_t s[32];
          tmem_load(s, lanes + buf * S::kRows + c);
          tmem_wait_load();
          tmem_loaded(s);
          sum_up(s, c);
        }
        const float2 total = halves(add2(sum2[0], sum2[1]));
        in_head += total.x + total.y;
        tc_fence_before();
        warp_arrive(s_empty(buf));
        warp_arrive(l_empty(stage));
        if (group == 0 && !known) look_up();
      }
      if (!ok) break;
      done += run;
      turn = (turn + run) % kGroups;
      in_keys += in_head;
      in_head = 0.f;
      if (!x.keys_end(run)) continue;
      // the key block's sums of all groups: the others hand theirs over
      if (group > 0) {
        if (f >= 2 && !(ok = warp_wait(c_empty(f & 1), ((f >> 1) - 1) & 1, &gave_up))) break;
        cross[f & 1][group - 1][key] = in_keys;
        warp_arrive(c_full(f & 1));
      } else {
        if (!known) look_up();
        if (!(ok = warp_wait(c_full(f & 1), (f >> 1) & 1, &gave_up))) break;
        float got = in_keys;
#pragma unroll
        for (int g = 0; g < kGroups - 1; ++g) got += cross[f & 1][g][key];
        warp_arrive(c_empty(f & 1));
        const long long rest = x.rest(run);
        if (x.whole && rest == 0) {
          add_weight(w, place, old, got);
        } else {
          w.partials[(size_t)(2 * blockIdx.x + (x.whole ? 1 : 0)) * kKeys + key] = got;
          if (x.whole) {
            w.slots[blockIdx.x * kKeys + key] = place;
            note = (int)((rest + start.per - 1) / start.per);
          }
        }
        known = false;
      }
      in_keys = 0.f;
      ++f;
    }
    if (tid == 0) w.notes[blockIdx.x] = note;
  } else if (any && warp == 12) {
    // ---- the products, issued by one thread
    if (lane == 0) {
      const uint32_t idesc = instruction(t.width, false);
      const uint32_t k_lo0 = operand_lo(k_s, 16), q_lo0 = operand_lo(q_s, 16);
      int i = 0;
      for (int run; ok && !x.done(); x.next(run)) {
        run = x.run();
        const uint32_t k_lo = k_lo0 + k_ring.stage * (S::kKBytes / 16);
        ok = bar_wait(k_full(k_ring.stage), k_ring.round & 1, &gave_up);
        for (int r = 0; ok && r < run; ++r, ++i, q_ring.next()) {
          const int buf = i % kS;
          ok = bar_wait(q_full(q_ring.stage), q_ring.round & 1, &gave_up) && (i < kS || bar_wait(s_empty(buf), (i / kS - 1) & 1, &gave_up));
          if (!ok) break;
          tc_fence_after();
          const uint32_t q_lo = q_lo0 + q_ring.stage * (q_bytes / 16), s_at = tmem + buf * S::kRows;
#pragma unroll
          for (int k = 0; k < kD / 16; ++k)
            mma_two(s_at, k_lo + (k / 4) * 64 + (k % 4) * 2, page_tile_hi<kD>(), q_lo + (k / 4) * (t.width * 8) + (k % 4) * 2, kOperandHi, idesc, k > 0);
          tc_commit(s_full(i));
          tc_commit(q_empty(q_ring.stage));
        }
        if (!ok) break;
        tc_commit(k_empty(k_ring.stage));
        k_ring.next();
      }
    }
    __syncwarp();
  } else if (any && warp == 13) {
    // ---- K tiles: lane `box` copies its tokens' page or part of one
    const int n_box = kKeys / t.box, box = lane;
    bool new_keys = true;
    int page = 0, token = 0, live = 0, page_b = -1, page_kb = 0, page_next = 0, token_next = 0;
    // the page of this lane's box in a key block of the walk's request; looked up a key block ahead
    auto page_of = [&](int kb, int* token) {
      const int j = kb * kKeys + box * t.box, i = (int)quotient(j, p.by_page);
      *token = j - i * p.page_size;
      return kb < x.req.kb1 && box < n_box && j < x.req.ctx + x.req.n ? p.table[(size_t)x.b * p.table_stride + i] : -1;
    };
    for (int run; ok && !x.done(); x.next(run)) {
      run = x.run();
      if (new_keys) {
        const int len = x.req.ctx + x.req.n;
        live = min(n_box, (len - x.kb * kKeys + t.box - 1) / t.box);
        if (page_b == x.b && page_kb == x.kb) {
          page = page_next;
          token = token_next;
        } else {
          page = page_of(x.kb, &token);
        }
        page_next = page_of(x.kb + 1, &token_next);
        page_b = x.b;
        page_kb = x.kb + 1;
      }
      const int stage = k_ring.stage;
      if (k_ring.round > 0 && !(ok = warp_wait(k_empty(stage), (k_ring.round - 1) & 1, &gave_up))) break;
      if (lane == 0) bar_expect(k_full(stage), (uint32_t)live * t.box * kD * 2);
      __syncwarp();
#ifdef GDN_TEST_HOOKS
      const bool issue = sent > 0 || (int)blockIdx.x != g_test_drop_block;
#else
      constexpr bool issue = true;
#endif
      if (issue && box < live) {
        // a page outside the pool: zeros; its tokens take no weight
        copy_page<kD>(&k_map, t.k_pages, k_s + stage * S::kKBytes + (uint32_t)(box * t.box * kD * 2), k_full(stage), t.box, token, x.h, page, p.n_pages);
      }
      ++sent;
      k_ring.next();
      new_keys = x.keys_end(run);
    }
  } else if (any && warp == 14) {
    // ---- Q tiles: lane c copies 64 columns
    const int rows = w.tokens * w.heads;
    for (int run; ok && !x.done(); x.next(run)) {
      run = x.run();
      for (int r = 0; r < run; ++r) {
        const int stage = q_ring.stage;
        if (q_ring.round > 0 && !(ok = warp_wait(q_empty(stage), (q_ring.round - 1) & 1, &gave_up))) break;
        if (lane == 0) bar_expect(q_full(stage), (uint32_t)rows * kD * 2);
        __syncwarp();
        if (lane < kChunks)
          tma_rows(&q_map, q_s + stage * q_bytes + lane * (t.width * 128), q_full(stage), lane * 64, x.h * p.G + x.head(x.m + r),
                   x.req.row0 + x.token(x.m + r));
        ++sent;
        q_ring.next();
      }
    }
  } else if (any && warp == 15) {
    // ---- the tiles' lse, in the exponent of 2 and negative: lane c takes columns c, c + 32, ..., whose tokens and heads are the
    // same in every tile; the next tile's are on their way while a place in the ring is waited for
    constexpr int kEach = S::kRows / 32;
    int64_t off[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int c = lane + 32 * k, token = (int)quotient(c, w.by_heads);
      off[k] = (int64_t)token * w.lse_row + c - token * w.heads;
    }
    auto load = [&](float (&v)[kEach], int m) {
      const int n_cols = x.columns(m);
      const float* const from = w.lse + (int64_t)(x.req.row0 + x.token(m)) * w.lse_row + x.h * p.G + x.head(m);
#pragma unroll
      for (int k = 0; k < kEach; ++k) v[k] = lane + 32 * k < n_cols ? __ldg(from + off[k]) : 0.f;
    };
    float now[kEach], ahead[kEach];
    int run = x.run(), r = 0;
    load(now, x.m);
    for (int i = 0; ok; ++i) {
      if (++r == run) {
        x.next(run);
        run = x.run();
        r = 0;
      }
      const bool more = !x.done();
      if (more) load(ahead, x.m + r);
      const int stage = i % kL;
      if (i >= kL && !(ok = warp_wait(l_empty(stage), (i / kL - 1) & 1, &gave_up))) break;
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        lse_s[stage][lane + 32 * k] = now[k] * -1.4426950408889634f;
        now[k] = ahead[k];
      }
      warp_arrive(l_full(i));
      if (!more) break;
    }
  }
  if (!any && tid == 0) w.notes[blockIdx.x] = 0;
  __syncthreads();
  if (gave_up) {
    // products and copies that may still be in flight, with a bound again
    const unsigned long long end = now_ns() + kWaitNs;
    if (tid == 12 * 32) {
      tc_commit(drained);
      while (!bar_try(drained, 0) && now_ns() < end) {
      }
    }
    if (lane == 0 && (warp == 13 || warp == 14)) {
      const int stages = warp == 13 ? t.n_k : t.n_q;
      for (int i = max(0, sent - stages); i < sent; ++i)
        while (!bar_try((warp == 13 ? k_full(0) : q_full(0)) + 8 * (i % stages), (i / stages) & 1) && now_ns() < end) {
        }
    }
    if (tid == 0) {
      w.notes[blockIdx.x] = 0;
      if (p.status) atomicOr(p.status, GDN_STATUS_TIMEOUT);
    }
    __syncthreads();
  }
  if (warp == 12) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// rows of q as [d][H_q][n_q_rows]
bool make_row_map(CUtensorMap* map, const WeightParams& w) {
  const EncodeFn encode = encoder();
  if (!encode) return false;
  const Params& p = w.p;
  const cuuint64_t H_q = (cuuint64_t)p.H_kv * p.G, dims[3] = {(cuuint64_t)p.d, H_q, (cuuint64_t)p.n_q_rows};
  // the stride of a dimension of one entry is never used, but must be a valid one
  const cuuint64_t head = (cuuint64_t)(H_q > 1 ? p.q_head : p.d) * 2, row = p.n_q_rows > 1 ? (cuuint64_t)p.q_row * 2 : head;
  const cuuint64_t strides[2] = {head, row};
  const cuuint32_t box[3] = {64, (cuuint32_t)w.heads, (cuuint32_t)w.tokens}, steps[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p.q), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kD>
int run(WeightTcParams& t, cudaStream_t st) {
  using S = WeightShape<kD>;
  if (cudaFuncSetAttribute(weight_tc_kernel<kD>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem) != cudaSuccess) return GDN_ERR_LAUNCH;
  set_weight_tiles(t.w, S::kRows);
  t.width = (t.w.tokens * t.w.heads + 15) / 16 * 16;
  // a step's few rows leave K to stream through: one stage more in flight
  const int q_bytes = t.width * kD * 2, least = S::kLeastK + (kD == 128 && t.width < S::kRows ? 1 : 0), left = S::kBytes - least * S::kKBytes;
  t.n_q = left / q_bytes < S::kMostQ ? left / q_bytes : S::kMostQ;
  t.n_k = (S::kBytes - t.n_q * q_bytes) / S::kKBytes;
  if (t.n_k > S::kMostK) t.n_k = S::kMostK;
  t.box = 16;
  while (t.box * 2 <= kWeightKeys && t.w.p.page_size % (t.box * 2) == 0) t.box *= 2;
  CUtensorMap k_map, q_map;
  if (!make_page_map(&k_map, &t.k_pages, t.w.p, t.w.p.k, t.w.p.k_token, t.w.p.k_head, t.w.p.k_page, t.box) || !make_row_map(&q_map, t.w))
    return GDN_ERR_LAUNCH;
  const int rc = launch(weight_tc_kernel<kD>, dim3(kWeightBlocks), dim3(kWeightThreads), S::kSmem, st, t, k_map, q_map);
  return rc != GDN_OK ? rc : launch_weight_join<kWeightKeys>(t.w, st);
}

size_t weight_tc_work() { return weight_work(kWeightBlocks, kWeightKeys); }

int run_weight_tc(WeightParams& w, void* work, cudaStream_t st) {
  set_weight_work(w, kWeightBlocks, kWeightKeys, work);
  WeightTcParams t{w, 0, 0, 0, 0, {0, 0}};
  return w.p.d == 64 ? run<64>(t, st) : w.p.d == 128 ? run<128>(t, st) : run<256>(t, st);
}

}  // namespace gdnattn

#ifdef GDN_TEST_HOOKS
// Test builds only: drop the first K copy of block `block` of later calls (-1 restores it).
extern "C" GDN_API int gdn_test_drop_weight_copy(int block) {
  return cudaMemcpyToSymbol(gdnattn::g_test_drop_block, &block, sizeof(int)) == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}
#endif
