// Attention of a request's new tokens over its pages in 32 bits, on the CUDA cores: the kernel, for gdn_paged_attention and
// gdn_shared_attention.
//
// simt_kernel: one pass over K and V with the running maximum and sum of the
//   softmax, 32-bit arithmetic throughout.  A block of four warps holds up to 32
//   rows (token, query head) of one kv head and walks blocks of 32 keys staged in
//   shared memory.  Scores: a lane is a key, a warp's rows (every fourth) in
//   registers; the row of K it reads is padded by four words so that the 16-byte
//   reads of a quarter warp fall into different banks, q is broadcast.  Output: a
//   lane owns d/32 columns of the warp's rows.  A warp computes 1, 2, 4 or 8 rows,
//   as few as the tile needs (64 requests of one token over 4000, 4 rows a head:
//   907 us, with 8 rows a warp throughout 1549).  K and V are copied asynchronously,
//   each under the other's products (436 us, copies waited for 907).
//   With few rows that case runs at 4.8 TB/s, 0.71 of a copy's rate: four block
//   barriers for each 32 keys, and no more than a block of K and one of V on their
//   way.  With many rows shared memory is the bound: eight rows of a warp take nine
//   16-byte reads (12 wavefronts) for 32 multiply-adds, 48 clocks of the SM's for the
//   four warps' 32 (a 4096-token prefill at d = 128: 4.5 ms, 30 TFLOP/s of some 76).
#pragma once
#include <type_traits>

#include "attn_common.cuh"

namespace gdnattn {

constexpr int kSimtRows = 32, kSimtKeys = 32, kSimtThreads = 128;
constexpr int kSimtMinUnits = 1;  // a block's least share: 3 requests of up to 700 tokens take 12.3 us, with 2 15.1, with 4 15.4

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }

template <int kD>
constexpr int simt_smem() {
  return (kSimtRows * kD + kSimtKeys * (kD + 4) + kSimtKeys * kD + kSimtRows * kSimtKeys) * (int)sizeof(float);
}

// kShared: the lines of gdn_shared_attention in place of requests, a tile's first part left in `dense` for its rows' join
template <int kD, bool kShared>
__global__ void __launch_bounds__(kSimtThreads, kD == 256 ? 2 : 3)
    simt_kernel(const Params p, const std::conditional_t<kShared, SharedParams, Nothing> sp) {
  constexpr int kR = kSimtRows, kN = kSimtKeys, kCols = kD / 32, kChunks = kD / 4;
  extern __shared__ float4 smem4[];
  float* const qs = reinterpret_cast<float*>(smem4);  // [kR][kD]
  float* const ks = qs + kR * kD;                     // [kN][kD + 4]
  float* const vs = ks + kN * (kD + 4);               // [kN][kD]
  float* const ps = vs + kN * kD;                     // [kR][kN]
  using W = Walk<kR, kN, kShared>;
  __shared__ long long scan[(kShared ? 3 : 1) * kSimtThreads / 32];
  __shared__ StartOf<typename W::R> start;
  __shared__ int row_at[kShared ? kR : 1];  // the tile's rows' rows of q and o
  __shared__ int64_t k_at[kN], v_at[kN];  // element offsets of the block's keys; -1: no key
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Lines lines = {};
  if constexpr (kShared)
    lines = find_lines<kR, kN, kSimtThreads>(p, sp, kSimtMinUnits, reinterpret_cast<int*>(ps + kR * kN), scan, &start);
  else
    find_start<kR, kN, kSimtThreads>(p, kSimtMinUnits, scan, &start);
  const auto s = start;
  int4 note = {0, 0, 0, 0};
  W w;
  if constexpr (kShared) {
    w.lines = &lines;
    w.align = sp.key_align;
  }
  auto segment = [&](auto warp_rows, int rows) {
      constexpr int kWarpRows = decltype(warp_rows)::value;
      __syncthreads();
      if constexpr (kShared) {
        if (tid < rows) row_at[tid] = lines.row_of(p, w.req, (int)quotient(w.m * kR + tid, p.by_G));
        __syncthreads();
      }
      for (int i = tid; i < 4 * kWarpRows * kChunks; i += kSimtThreads) {
        const int r = i / kChunks, c = i % kChunks, at = w.m * kR + r;
        float4 x = {0.f, 0.f, 0.f, 0.f};
        if (r < rows) {
          int q_row;
          if constexpr (kShared) q_row = row_at[r];
          else q_row = w.req.row0 + at / p.G;
          x = load4(static_cast<const float*>(p.q) + q_row * p.q_row + (w.h * p.G + at % p.G) * p.q_head + 4 * c);
        }
        reinterpret_cast<float4*>(qs)[i] = x;
      }
      float top[kWarpRows], sum[kWarpRows], acc[kWarpRows][kCols];
      int last[kWarpRows];  // the last position a row sees
#pragma unroll
      for (int r = 0; r < kWarpRows; ++r) {
        top[r] = -INFINITY;
        sum[r] = 0.f;
        last[r] = w.req.last((int)quotient(w.m * kR + r * 4 + warp, p.by_G));
#pragma unroll
        for (int c = 0; c < kCols; ++c) acc[r][c] = 0.f;
      }
      // a key's place in the caches, found a block ahead by the first kN threads
      const int len = w.req.len(), first_key = w.first_key();
      const int32_t* const pages = p.table + (size_t)w.table_row() * p.table_stride;
      auto page_of = [&](int j) { return j < len ? pages[quotient(first_key + j, p.by_page)] : -1; };
      auto place = [&](int j, int page) {
        const bool good = (unsigned)page < (unsigned)p.n_pages;
        const int token = first_key + j - (int)quotient(first_key + j, p.by_page) * p.page_size;
        k_at[tid] = good ? page * p.k_page + w.h * p.k_head + token * p.k_token : -1;
        v_at[tid] = good ? page * p.v_page + w.h * p.v_head + token * p.v_token : -1;
        if (!good && j < len && p.status) atomicOr(p.status, GDN_STATUS_BAD_PAGE);
      };
      auto fetch = [&](float* to, int stride, const void* from, const int64_t* at) {
#pragma unroll 4
        for (int i = tid; i < kN * kChunks; i += kSimtThreads) {
          const int j = i / kChunks, c = i % kChunks;
          const int64_t off = at[j];
          copy16(to + j * stride + 4 * c, static_cast<const float*>(from) + (off >= 0 ? off + 4 * c : 0), off >= 0);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      if (tid < kN) place(w.kb0 * kN + tid, page_of(w.kb0 * kN + tid));
      __syncthreads();
      fetch(ks, kD + 4, p.k, k_at);
      fetch(vs, kD, p.v, v_at);
      for (int kb = w.kb0; kb < w.kb1; ++kb) {
        const bool more = kb + 1 < w.kb1;
        const int ahead = (kb + 1) * kN + tid;
        const int page = more && tid < kN ? page_of(ahead) : -1;
        asm volatile("cp.async.wait_group 1;" ::: "memory");  // K; V may still be on its way
        __syncthreads();
        float sc[kWarpRows] = {};
#pragma unroll 4
        for (int c = 0; c < kChunks; ++c) {
          const float4 kx = *reinterpret_cast<const float4*>(ks + lane * (kD + 4) + 4 * c);
#pragma unroll
          for (int r = 0; r < kWarpRows; ++r) {
            const float4 qx = *reinterpret_cast<const float4*>(qs + (r * 4 + warp) * kD + 4 * c);
            sc[r] = fmaf(qx.x, kx.x, sc[r]);
            sc[r] = fmaf(qx.y, kx.y, sc[r]);
            sc[r] = fmaf(qx.z, kx.z, sc[r]);
            sc[r] = fmaf(qx.w, kx.w, sc[r]);
          }
        }
        const int j = kb * kN + lane;
#pragma unroll
        for (int r = 0; r < kWarpRows; ++r) {
          const float x = j <= last[r] ? sc[r] * p.scale_log2 : -INFINITY;
          float m = x;
#pragma unroll
          for (int off = 16; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, off));
          m = fmaxf(m, top[r]);
          const float base = m == -INFINITY ? 0.f : m;  // no key yet: exp2(-inf - 0) = 0
          const float shrink = exp2f(top[r] - base), e = exp2f(x - base);
          top[r] = m;
          sum[r] = sum[r] * shrink + e;  // this lane's share
#pragma unroll
          for (int c = 0; c < kCols; ++c) acc[r][c] *= shrink;
          ps[(r * 4 + warp) * kN + lane] = e;
        }
        if (more && tid < kN) place(ahead, page);
        __syncthreads();
        if (more) fetch(ks, kD + 4, p.k, k_at);
        else asm volatile("cp.async.commit_group;" ::: "memory");
        asm volatile("cp.async.wait_group 1;" ::: "memory");  // V
        __syncthreads();
#pragma unroll 2
        for (int j4 = 0; j4 < kN; j4 += 4) {
          float vx[4][kCols];
#pragma unroll
          for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int c = 0; c < kCols / 2; ++c) {
              const float2 x = *reinterpret_cast<const float2*>(vs + (j4 + u) * kD + (c * 32 + lane) * 2);
              vx[u][2 * c] = x.x;
              vx[u][2 * c + 1] = x.y;
            }
#pragma unroll
          for (int r = 0; r < kWarpRows; ++r) {
            const float4 e = *reinterpret_cast<const float4*>(ps + (r * 4 + warp) * kN + j4);
            const float es[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
              for (int c = 0; c < kCols; ++c) acc[r][c] = fmaf(es[u], vx[u][c], acc[r][c]);
          }
        }
        __syncthreads();
        if (more) fetch(vs, kD, p.v, v_at);
      }
      bool joins = false;  // the tile's rows have parts over a prefix and over their own keys
      if constexpr (kShared) joins = w.req.prefix != 0;
      const bool whole = w.kb0 == 0 && w.kb1 == w.blocks && !joins, first = joins && w.kb0 == 0;
      const int slot = w.kb0 == 0 ? 1 : 0;
      if (!whole && !first && slot == 1) note = note_of(w, s);
      float* const part = partial(p, blockIdx.x, slot, kR);
#pragma unroll
      for (int r = 0; r < kWarpRows; ++r) {
        float l = sum[r];
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) l += __shfl_xor_sync(kFull, l, off);
        const int row = r * 4 + warp, at = w.m * kR + row;
        if (row >= rows) continue;
        int o_row;
        const int head = w.h * p.G + at % p.G;
        float* out = part + row * kD;  // this row's parts
        float2* out_stats = reinterpret_cast<float2*>(part + kR * kD) + row;
        if constexpr (kShared) {
          o_row = row_at[row];
          if (first) {
            const size_t place = place_of(p, sp, !w.req.flat(), lines.rank_of(w.req, at / p.G), w.h, at % p.G);
            out = sp.dense + place * kD;
            out_stats = reinterpret_cast<float2*>(sp.entries + place);
            if (lane == 0) reinterpret_cast<int2*>(out_stats)[1] = make_int2(blockIdx.x, entry_word(followers_of(w, s), row));
          }
          if (lane == 0 && whole && sp.lse) sp.lse[(int64_t)o_row * sp.lse_row + head] = (top[r] + log2f(l)) * kLn2;
        } else {
          o_row = w.req.row0 + at / p.G;
        }
        if (whole) {
          const float inv = 1.f / l;
          float* dst = static_cast<float*>(p.o) + o_row * p.o_row + head * p.o_head;
#pragma unroll
          for (int c = 0; c < kCols / 2; ++c) {
            const int col = (c * 32 + lane) * 2;
            const float x = acc[r][2 * c] * inv, y = acc[r][2 * c + 1] * inv;
            *reinterpret_cast<float2*>(dst + col) = make_float2(x, y);
          }
        } else {
#pragma unroll
          for (int c = 0; c < kCols / 2; ++c)
            *reinterpret_cast<float2*>(out + (c * 32 + lane) * 2) = make_float2(acc[r][2 * c], acc[r][2 * c + 1]);
          if (lane == 0) *out_stats = make_float2(top[r], l);
        }
      }
  };
  if (begin(w, p, s)) {
    for (; !w.done(); w.next()) {
      const int rows = (int)min((long long)kR, (long long)w.req.n * p.G - (long long)w.m * kR);
      if (rows <= 4) segment(std::integral_constant<int, 1>(), rows);
      else if (rows <= 8) segment(std::integral_constant<int, 2>(), rows);
      else if (rows <= 16) segment(std::integral_constant<int, 4>(), rows);
      else segment(std::integral_constant<int, 8>(), rows);
    }
  }
  if (tid == 0) p.notes[blockIdx.x] = note;
}

// blocks of the launch: a fixed number per d and type (as many as 152 SMs hold
// at once), so that the work buffer's size depends on neither lengths nor device
constexpr int kSms = 152;
constexpr int simt_blocks(int d) { return kSms * (d == 256 ? 2 : 3); }

// Launches the attention and the join of its parts.
template <int kD, bool kShared>
int run_simt(Params p, const std::conditional_t<kShared, SharedParams, Nothing>& sp, cudaStream_t st) {
  size_t smem = simt_smem<kD>(), most = smem;
  if constexpr (kShared) {
    smem += sizeof(int) * lines_words(p.B, sp.n_groups);
    most += sizeof(int) * kMaxLinesWords;
  }
  if (most > 48 * 1024 &&
      cudaFuncSetAttribute(simt_kernel<kD, kShared>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most) != cudaSuccess)
    return GDN_ERR_LAUNCH;
  p.n_blocks = simt_blocks(kD);
  const int rc = launch(simt_kernel<kD, kShared>, dim3(p.n_blocks), dim3(kSimtThreads), smem, st, p, sp);
  if (rc != GDN_OK) return rc;
  if constexpr (kShared) return launch_combine_shared<float, kD, kSimtRows>(p, sp, st);
  else return launch(combine_kernel<float, kD, kSimtRows>, dim3(p.n_blocks, 4), dim3(32 * kCombineWarps), 0, st, p);
}

template <bool kShared>
int run_simt(const Params& p, const std::conditional_t<kShared, SharedParams, Nothing>& sp, cudaStream_t st) {
  return p.d == 64 ? run_simt<64, kShared>(p, sp, st) : p.d == 128 ? run_simt<128, kShared>(p, sp, st) : run_simt<256, kShared>(p, sp, st);
}

}  // namespace gdnattn
