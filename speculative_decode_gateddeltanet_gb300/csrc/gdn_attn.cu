// Attention of a request's new tokens over its pages: argument checks, the
// launch, and the 32-bit kernel, on the CUDA cores.
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
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "attn_common.cuh"
#include "attn_tc.h"

namespace gdnattn {

constexpr int kSimtRows = 32, kSimtKeys = 32, kSimtThreads = 128;
constexpr int kSimtMinUnits = 1;  // a block's least share: 3 requests of up to 700 tokens take 12.3 us, with 2 15.1, with 4 15.4

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// 16 bytes into shared memory, or zeros
__device__ __forceinline__ void copy16(float* to, const float* from, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from), "r"(valid ? 16 : 0) : "memory");
}

template <int kD>
constexpr int simt_smem() {
  return (kSimtRows * kD + kSimtKeys * (kD + 4) + kSimtKeys * kD + kSimtRows * kSimtKeys) * (int)sizeof(float);
}

template <int kD>
__global__ void __launch_bounds__(kSimtThreads, kD == 256 ? 2 : 3) simt_kernel(const Params p) {
  constexpr int kR = kSimtRows, kN = kSimtKeys, kCols = kD / 32, kChunks = kD / 4;
  extern __shared__ float4 smem4[];
  float* const qs = reinterpret_cast<float*>(smem4);  // [kR][kD]
  float* const ks = qs + kR * kD;                     // [kN][kD + 4]
  float* const vs = ks + kN * (kD + 4);               // [kN][kD]
  float* const ps = vs + kN * kD;                     // [kR][kN]
  __shared__ long long scan[kSimtThreads / 32];
  __shared__ Start start;
  __shared__ int64_t k_at[kN], v_at[kN];  // element offsets of the block's keys; -1: no key
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  find_start<kR, kN, kSimtThreads>(p, kSimtMinUnits, scan, &start);
  const Start s = start;
  int4 note = {0, 0, 0, 0};
  Walk<kR, kN> w;
  auto segment = [&](auto warp_rows, int rows) {
      constexpr int kWarpRows = decltype(warp_rows)::value;
      __syncthreads();
      for (int i = tid; i < 4 * kWarpRows * kChunks; i += kSimtThreads) {
        const int r = i / kChunks, c = i % kChunks, at = w.m * kR + r;
        float4 x = {0.f, 0.f, 0.f, 0.f};
        if (r < rows)
          x = load4(static_cast<const float*>(p.q) + (w.req.row0 + at / p.G) * p.q_row + (w.h * p.G + at % p.G) * p.q_head + 4 * c);
        reinterpret_cast<float4*>(qs)[i] = x;
      }
      float top[kWarpRows], sum[kWarpRows], acc[kWarpRows][kCols];
      int last[kWarpRows];  // the last position a row sees
#pragma unroll
      for (int r = 0; r < kWarpRows; ++r) {
        top[r] = -INFINITY;
        sum[r] = 0.f;
        last[r] = w.req.ctx + (int)quotient(w.m * kR + r * 4 + warp, p.by_G);
#pragma unroll
        for (int c = 0; c < kCols; ++c) acc[r][c] = 0.f;
      }
      // a key's place in the caches, found a block ahead by the first kN threads
      const int len = w.req.ctx + w.req.n;
      const int32_t* const pages = p.table + (size_t)w.b * p.table_stride;
      auto page_of = [&](int j) { return j < len ? pages[quotient(j, p.by_page)] : -1; };
      auto place = [&](int j, int page) {
        const bool good = (unsigned)page < (unsigned)p.n_pages;
        const int token = j - (int)quotient(j, p.by_page) * p.page_size;
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
      const bool whole = w.kb0 == 0 && w.kb1 == w.blocks;
      const int slot = w.kb0 == 0 ? 1 : 0;
      if (!whole && slot == 1) note = note_of(w, s);
      float* const out = partial(p, blockIdx.x, slot, kR);
#pragma unroll
      for (int r = 0; r < kWarpRows; ++r) {
        float l = sum[r];
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) l += __shfl_xor_sync(kFull, l, off);
        const int row = r * 4 + warp, at = w.m * kR + row;
        if (row >= rows) continue;
        if (whole) {
          const float inv = 1.f / l;
          float* dst = static_cast<float*>(p.o) + (w.req.row0 + at / p.G) * p.o_row + (w.h * p.G + at % p.G) * p.o_head;
#pragma unroll
          for (int c = 0; c < kCols / 2; ++c) {
            const int col = (c * 32 + lane) * 2;
            const float x = acc[r][2 * c] * inv, y = acc[r][2 * c + 1] * inv;
            *reinterpret_cast<float2*>(dst + col) = make_float2(x, y);
          }
        } else {
#pragma unroll
          for (int c = 0; c < kCols / 2; ++c)
            *reinterpret_cast<float2*>(out + row * kD + (c * 32 + lane) * 2) = make_float2(acc[r][2 * c], acc[r][2 * c + 1]);
          if (lane == 0) reinterpret_cast<float2*>(out + kR * kD)[row] = make_float2(top[r], l);
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

int blocks_of(int d, int dtype) { return dtype == GDN_DTYPE_BF16 ? tc_blocks() : simt_blocks(d); }

size_t work_bytes(int d, int dtype) {
  const size_t blocks = blocks_of(d, dtype), rows = dtype == GDN_DTYPE_BF16 ? tc_rows() : kSimtRows;
  return blocks * sizeof(int4) + blocks * 2 * rows * (d + 2) * sizeof(float);
}

template <int kD>
int run_simt(Params& p, cudaStream_t st) {
  constexpr int smem = simt_smem<kD>();
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(simt_kernel<kD>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return GDN_ERR_LAUNCH;
  p.n_blocks = simt_blocks(kD);
  const int rc = launch(simt_kernel<kD>, dim3(p.n_blocks), dim3(kSimtThreads), smem, st, p);
  if (rc != GDN_OK) return rc;
  return launch(combine_kernel<float, kD, kSimtRows>, dim3(p.n_blocks, 4), dim3(32 * kCombineWarps), 0, st, p);
}

int run_simt(Params& p, cudaStream_t st) {
  return p.d == 64 ? run_simt<64>(p, st) : p.d == 128 ? run_simt<128>(p, st) : run_simt<256>(p, st);
}

int check_sizes(const gdn_paged_attn_args* a) {
  if (!a) return GDN_ERR_INVALID_ARG;
  if (a->B < 0 || a->R < 0 || a->H_kv < 1 || a->H_q < 1 || a->page_size < 1 || a->n_pages < 1 || a->max_pages < 0 ||
      a->table_stride < a->max_pages || a->n_q_rows < 0)
    return GDN_ERR_INVALID_ARG;
  if (a->in_dtype != GDN_DTYPE_BF16 && a->in_dtype != GDN_DTYPE_F32) return GDN_ERR_UNSUPPORTED;
  if ((a->d != 64 && a->d != 128 && a->d != 256) || a->H_q % a->H_kv != 0 || a->H_q / a->H_kv > 128 ||
      (int64_t)a->n_pages * a->page_size > INT32_MAX || (int64_t)a->B * a->R > INT32_MAX)
    return GDN_ERR_UNSUPPORTED;
  if (a->in_dtype == GDN_DTYPE_BF16 && (a->page_size % 16 != 0 || a->page_size > 1024)) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

float scale_log2(const gdn_paged_attn_args* a) { return (float)((double)a->scale * 1.4426950408889634); }

int check(const gdn_paged_attn_args* a) {
  const int rc = check_sizes(a);
  if (rc != GDN_OK) return rc;
  if (!(a->scale - a->scale == 0.f)) return GDN_ERR_INVALID_ARG;  // not finite
  if (!std::isfinite(scale_log2(a))) return GDN_ERR_UNSUPPORTED;
  if (a->B == 0 || a->n_q_rows == 0) return GDN_OK;
  if (!a->q || !a->k_cache || !a->v_cache || !a->block_table || !a->ctx_len || !a->n_rows || !a->o || !a->work)
    return GDN_ERR_INVALID_ARG;
  if (a->R == 0 && !a->row_start) return GDN_ERR_INVALID_ARG;
  const int size = a->in_dtype == GDN_DTYPE_BF16 ? 2 : 4;
  const int64_t strides[] = {a->q_row_stride, a->q_head_stride, a->k_page_stride, a->k_head_stride, a->k_token_stride,
                             a->v_page_stride, a->v_head_stride, a->v_token_stride, a->o_row_stride, a->o_head_stride};
  for (int64_t s : strides)
    if (s * size % 16 != 0) return GDN_ERR_MISALIGNED;
  for (int i = 2; i < 8; ++i)  // the pools': a negative offset is a key that is not there
    if (strides[i] < 0) return GDN_ERR_INVALID_ARG;
  auto al = [](const void* ptr, uintptr_t n) { return reinterpret_cast<uintptr_t>(ptr) % n == 0; };
  if (!al(a->q, 16) || !al(a->k_cache, 16) || !al(a->v_cache, 16) || !al(a->o, 16) || !al(a->work, 16) ||
      !al(a->block_table, 4) || !al(a->ctx_len, 4) || !al(a->n_rows, 4) || !al(a->row_start, 4) || !al(a->status, 4))
    return GDN_ERR_MISALIGNED;
  return GDN_OK;
}

}  // namespace gdnattn

using namespace gdnattn;

extern "C" GDN_API size_t gdn_paged_attention_work_bytes(const gdn_paged_attn_args* args) {
  return check_sizes(args) == GDN_OK ? work_bytes(args->d, args->in_dtype) : 0;
}

extern "C" GDN_API int gdn_paged_attention(const gdn_paged_attn_args* a, void* stream) {
  const int rc = check(a);
  if (rc != GDN_OK || a->B == 0 || a->n_q_rows == 0) return rc;
  Params p;
  p.B = a->B;
  p.R = a->R;
  p.H_kv = a->H_kv;
  p.G = a->H_q / a->H_kv;
  p.d = a->d;
  p.page_size = a->page_size;
  p.n_pages = a->n_pages;
  p.table_stride = a->table_stride;
  p.n_q_rows = a->n_q_rows;
  p.max_tokens = (int)std::min((int64_t)a->max_pages * a->page_size, (int64_t)kMaxIndex);
  p.max_rows = kMaxIndex / p.G;
  p.scale_log2 = scale_log2(a);
  p.by_G = make_div((uint32_t)p.G);
  p.by_page = make_div((uint32_t)p.page_size);
  p.q = a->q;
  p.q_row = a->q_row_stride;
  p.q_head = a->q_head_stride;
  p.k = a->k_cache;
  p.k_page = a->k_page_stride;
  p.k_head = a->k_head_stride;
  p.k_token = a->k_token_stride;
  p.v = a->v_cache;
  p.v_page = a->v_page_stride;
  p.v_head = a->v_head_stride;
  p.v_token = a->v_token_stride;
  p.table = a->block_table;
  p.ctx_len = a->ctx_len;
  p.n_rows = a->n_rows;
  p.row_start = a->row_start;
  p.o = a->o;
  p.o_row = a->o_row_stride;
  p.o_head = a->o_head_stride;
  p.status = a->status;
  p.notes = static_cast<int4*>(a->work);
  p.partials = reinterpret_cast<float*>(p.notes + blocks_of(p.d, a->in_dtype));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return a->in_dtype == GDN_DTYPE_BF16 ? run_tc(p, st) : run_simt(p, st);
}
