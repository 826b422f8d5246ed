// gdn_attn_weight: argument checks, the launches, and the 32-bit kernel, on the CUDA cores.
//
// weight_simt_kernel: a block holds 64 keys and up to 32 rows in shared memory and computes their 2048 products in 32 bits: a
//   thread has two keys and four rows, whose sums over rows, tiles and heads stay in its registers until the block of keys is
//   done; then the eight warps' sums are added in warp order.  Two blocks an SM, each of which waits for its copies while the
//   other computes.  Bound by shared memory where rows are many (six 16-byte reads for 32 multiply-adds), by the copies'
//   latency where they are few.  Measured: 16 requests of 4 tokens over 1000 to 8000 at d = 256 117 us (1.3 TB/s), 2048 prompt
//   tokens of 16 heads at d = 128 724 us (24 TFLOP/s), three short requests at d = 64 8.0 us.
#include <algorithm>
#include <cmath>

#include "weight_common.cuh"

namespace gdnattn {

constexpr int kWsThreads = 256, kWsKeys = 64, kWsRows = 32, kWsBlocks = 304;

template <int kD>
constexpr int weight_simt_smem() {
  return (kWsKeys + kWsRows) * (kD + 4) * (int)sizeof(float);
}

template <int kD>
__global__ void __launch_bounds__(kWsThreads, 2) weight_simt_kernel(const WeightParams w) {
  constexpr int kPitch = kD + 4, kChunks = kD / 4;
  extern __shared__ float4 smem4[];
  float* const ks = reinterpret_cast<float*>(smem4);  // [kWsKeys][kPitch]
  float* const qs = ks + kWsKeys * kPitch;            // [kWsRows][kPitch]
  __shared__ long long scan[kWsThreads / 32];
  __shared__ WeightStart start;
  __shared__ int64_t k_at[kWsKeys];  // element offsets of the keys of head 0; -1: no key
  __shared__ float lse_s[kWsRows], cross[kWsThreads / 32][kWsKeys];
  pdl_wait();
  pdl_trigger();
  const Params& p = w.p;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  find_weight_start<kWsKeys, kWsThreads>(w, scan, &start);
  int note = 0;
  WeightWalk<kWsKeys> x;
  float in_keys[2] = {0.f, 0.f}, in_head[2] = {0.f, 0.f};
  bool new_head = true, new_keys = true;
  if (x.begin(w, start)) {
    for (; !x.done(); x.next(1)) {
      __syncthreads();  // the last unit's products are done
      if (new_keys && tid < kWsKeys) {
        const int j = x.kb * kWsKeys + tid, i = (int)quotient(j, p.by_page);
        const int page = j < x.req.ctx + x.req.n ? p.table[(size_t)x.b * p.table_stride + i] : -1;
        k_at[tid] = (unsigned)page < (unsigned)p.n_pages ? page * p.k_page + (j - i * p.page_size) * p.k_token : -1;
      }
      const int n_cols = x.columns(x.m), head0 = x.h * p.G + x.head(x.m), row0 = x.req.row0 + x.token(x.m);
      for (int i = tid; i < kWsRows * kChunks; i += kWsThreads) {
        const int r = i / kChunks, c = i % kChunks, token = (int)quotient(r, w.by_heads);
        const bool valid = r < n_cols;
        copy16(qs + r * kPitch + 4 * c,
               static_cast<const float*>(p.q) + (valid ? (int64_t)(row0 + token) * p.q_row + (int64_t)(head0 + r - token * w.heads) * p.q_head + 4 * c : 0),
               valid);
      }
      if (tid < n_cols) {
        const int token = (int)quotient(tid, w.by_heads);
        lse_s[tid] = w.lse[(int64_t)(row0 + token) * w.lse_row + head0 + tid - token * w.heads];
      }
      if (new_head) {
        if (new_keys) __syncthreads();  // k_at
        for (int i = tid; i < kWsKeys * kChunks; i += kWsThreads) {
          const int j = i / kChunks, c = i % kChunks;
          const int64_t off = k_at[j];
          copy16(ks + j * kPitch + 4 * c, static_cast<const float*>(p.k) + (off >= 0 ? off + x.h * p.k_head + 4 * c : 0), off >= 0);
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncthreads();
      float s[2][4] = {};
      const int n_mine = min(4, (n_cols - warp + 7) / 8);  // rows warp, warp + 8, ...
      if (n_mine > 0) {
#pragma unroll 4
        for (int c = 0; c < kChunks; ++c) {
          const float4 k0 = *reinterpret_cast<const float4*>(ks + lane * kPitch + 4 * c);
          const float4 k1 = *reinterpret_cast<const float4*>(ks + (lane + 32) * kPitch + 4 * c);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            if (r >= n_mine) break;
            const float4 q = *reinterpret_cast<const float4*>(qs + (warp + 8 * r) * kPitch + 4 * c);
            s[0][r] = fmaf(k0.x, q.x, s[0][r]);
            s[0][r] = fmaf(k0.y, q.y, s[0][r]);
            s[0][r] = fmaf(k0.z, q.z, s[0][r]);
            s[0][r] = fmaf(k0.w, q.w, s[0][r]);
            s[1][r] = fmaf(k1.x, q.x, s[1][r]);
            s[1][r] = fmaf(k1.y, q.y, s[1][r]);
            s[1][r] = fmaf(k1.z, q.z, s[1][r]);
            s[1][r] = fmaf(k1.w, q.w, s[1][r]);
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int past = x.kb * kWsKeys + lane + 32 * k - x.req.ctx - x.token(x.m);  // rows from this token on see the key
          float sum = 0.f;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int row = warp + 8 * r;
            if (r < n_mine && (int)quotient(row, w.by_heads) >= past) sum += expf(fmaf(s[k][r], w.scale, -lse_s[row]));
          }
          in_head[k] += sum;
        }
      }
      new_head = x.run() == 1;
      new_keys = x.keys_end(1);
      if (new_head) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          in_keys[k] += in_head[k];
          in_head[k] = 0.f;
        }
      }
      if (!new_keys) continue;
      cross[warp][lane] = in_keys[0];
      cross[warp][lane + 32] = in_keys[1];
      in_keys[0] = in_keys[1] = 0.f;
      __syncthreads();
      if (tid < kWsKeys) {
        float got = 0.f;
#pragma unroll
        for (int i = 0; i < kWsThreads / 32; ++i) got += cross[i][tid];
        const long long rest = x.rest(1);
        if (!x.whole) {
          w.partials[(size_t)(2 * blockIdx.x) * kWsKeys + tid] = got;
        } else {
          const int place = weight_place(w, x.req, x.b, x.kb * kWsKeys + tid);
          if (rest == 0) {
            add_weight(w, place, old_weight(w, place), got);
          } else {
            w.partials[(size_t)(2 * blockIdx.x + 1) * kWsKeys + tid] = got;
            w.slots[blockIdx.x * kWsKeys + tid] = place;
            note = (int)((rest + start.per - 1) / start.per);
          }
        }
      }
    }
  }
  if (tid == 0) w.notes[blockIdx.x] = note;
}

template <int kD>
int run(const WeightParams& w, cudaStream_t st) {
  constexpr int smem = weight_simt_smem<kD>();
  if (cudaFuncSetAttribute(weight_simt_kernel<kD>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return GDN_ERR_LAUNCH;
  const int rc = launch(weight_simt_kernel<kD>, dim3(kWsBlocks), dim3(kWsThreads), smem, st, w);
  return rc != GDN_OK ? rc : launch_weight_join<kWsKeys>(w, st);
}

int run_weight_simt(WeightParams& w, void* work, cudaStream_t st) {
  set_weight_work(w, kWsBlocks, kWsKeys, work);
  set_weight_tiles(w, kWsRows);
  return w.p.d == 64 ? run<64>(w, st) : w.p.d == 128 ? run<128>(w, st) : run<256>(w, st);
}

// the attention's checks on what the two calls share
gdn_paged_attn_args as_attention(const gdn_attn_weight_args* a) {
  gdn_paged_attn_args t = {};
  t.B = a->B;
  t.R = a->R;
  t.H_q = a->H_q;
  t.H_kv = a->H_kv;
  t.d = a->d;
  t.page_size = a->page_size;
  t.n_pages = a->n_pages;
  t.max_pages = a->max_pages;
  t.table_stride = a->table_stride;
  t.n_q_rows = a->n_q_rows;
  t.in_dtype = a->in_dtype;
  t.scale = a->scale;
  t.q = a->q;
  t.q_row_stride = a->q_row_stride;
  t.q_head_stride = a->q_head_stride;
  t.k_cache = t.v_cache = a->k_cache;
  t.k_page_stride = t.v_page_stride = a->k_page_stride;
  t.k_head_stride = t.v_head_stride = a->k_head_stride;
  t.k_token_stride = t.v_token_stride = a->k_token_stride;
  t.block_table = a->block_table;
  t.ctx_len = a->ctx_len;
  t.n_rows = a->n_rows;
  t.row_start = a->row_start;
  t.o = a->work;  // nothing is written through it
  t.work = a->work;
  t.status = a->status;
  return t;
}

int check(const gdn_attn_weight_args* a) {
  if (!a) return GDN_ERR_INVALID_ARG;
  const gdn_paged_attn_args t = as_attention(a);
  const int rc = check(&t);
  if (rc != GDN_OK) return rc;
  if ((a->fresh != 0 && a->fresh != 1) || !std::isfinite(a->keep)) return GDN_ERR_INVALID_ARG;
  if (a->B == 0 || a->n_q_rows == 0) return GDN_OK;
  if (!a->lse || !a->weight || a->lse_row_stride < a->H_q || a->q_row_stride < 0 || a->q_head_stride < 0) return GDN_ERR_INVALID_ARG;
  if (a->in_dtype == GDN_DTYPE_BF16 && (!map_stride(a->q_row_stride, a->n_q_rows) || !map_stride(a->q_head_stride, a->H_q))) return GDN_ERR_UNSUPPORTED;
  auto al = [](const void* ptr) { return reinterpret_cast<uintptr_t>(ptr) % 4 == 0; };
  return al(a->lse) && al(a->first) && al(a->position) && al(a->weight) && al(a->born) ? GDN_OK : GDN_ERR_MISALIGNED;
}

}  // namespace gdnattn

using namespace gdnattn;

extern "C" GDN_API size_t gdn_attn_weight_work_bytes(const gdn_attn_weight_args* args) {
  if (!args) return 0;
  const gdn_paged_attn_args t = as_attention(args);
  return gdn_paged_attention_work_bytes(&t) ? (args->in_dtype == GDN_DTYPE_BF16 ? weight_tc_work() : weight_work(kWsBlocks, kWsKeys)) : 0;
}

extern "C" GDN_API int gdn_attn_weight(const gdn_attn_weight_args* a, void* stream) {
  const int rc = check(a);
  if (rc != GDN_OK || a->B == 0 || a->n_q_rows == 0) return rc;
  const gdn_paged_attn_args t = as_attention(a);
  WeightParams w = {};
  w.p = params_of(&t);
  w.scale = a->scale;
  w.keep = a->keep;
  w.fresh = a->fresh;
  w.lse = a->lse;
  w.lse_row = a->lse_row_stride;
  w.first = a->first;
  w.position = a->position;
  w.weight = a->weight;
  w.born = a->born;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return a->in_dtype == GDN_DTYPE_BF16 ? run_weight_tc(w, a->work, st) : run_weight_simt(w, a->work, st);
}
