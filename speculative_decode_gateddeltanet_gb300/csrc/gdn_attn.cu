// gdn_paged_attention: argument checks and the launch.
#include <algorithm>
#include <cmath>

#include "attn_simt.cuh"
#include "attn_tc.h"

namespace gdnattn {

int blocks_of(int d, int dtype) { return dtype == GDN_DTYPE_BF16 ? tc_blocks() : simt_blocks(d); }

size_t work_bytes(int d, int dtype) {
  const size_t blocks = blocks_of(d, dtype), rows = dtype == GDN_DTYPE_BF16 ? tc_rows() : kSimtRows;
  return blocks * sizeof(int4) + blocks * 2 * rows * (d + 2) * sizeof(float);
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
  if (a->in_dtype == GDN_DTYPE_BF16 &&
      (!map_stride(a->k_token_stride, a->page_size) || !map_stride(a->k_head_stride, a->H_kv) || !map_stride(a->k_page_stride, a->n_pages) ||
       !map_stride(a->v_token_stride, a->page_size) || !map_stride(a->v_head_stride, a->H_kv) || !map_stride(a->v_page_stride, a->n_pages)))
    return GDN_ERR_UNSUPPORTED;
  auto al = [](const void* ptr, uintptr_t n) { return reinterpret_cast<uintptr_t>(ptr) % n == 0; };
  if (!al(a->q, 16) || !al(a->k_cache, 16) || !al(a->v_cache, 16) || !al(a->o, 16) || !al(a->work, 16) ||
      !al(a->block_table, 4) || !al(a->ctx_len, 4) || !al(a->n_rows, 4) || !al(a->row_start, 4) || !al(a->status, 4))
    return GDN_ERR_MISALIGNED;
  return GDN_OK;
}

void set_work(Params& p, int dtype, void* work) {
  p.notes = static_cast<int4*>(work);
  p.partials = reinterpret_cast<float*>(p.notes + blocks_of(p.d, dtype));
}

Params params_of(const gdn_paged_attn_args* a) {
  Params p = {};
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
  return p;
}

}  // namespace gdnattn

using namespace gdnattn;

extern "C" GDN_API size_t gdn_paged_attention_work_bytes(const gdn_paged_attn_args* args) {
  return check_sizes(args) == GDN_OK ? work_bytes(args->d, args->in_dtype) : 0;
}

extern "C" GDN_API int gdn_paged_attention(const gdn_paged_attn_args* a, void* stream) {
  const int rc = check(a);
  if (rc != GDN_OK || a->B == 0 || a->n_q_rows == 0) return rc;
  Params p = params_of(a);
  set_work(p, a->in_dtype, a->work);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return a->in_dtype == GDN_DTYPE_BF16 ? run_tc(p, st) : run_simt<false>(p, Nothing{}, st);
}
