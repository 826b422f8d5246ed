// gdn_shared_attention: argument checks and the launches.
#include <algorithm>

#include "attn_simt.cuh"
#include "attn_tc.h"
#include "gdnlong.h"

namespace gdnattn {

int check_sizes(const gdn_shared_attn_args* a) {
  if (!a || a->n_groups < 0 || a->reserved != 0) return GDN_ERR_INVALID_ARG;
  if (a->attn.B > kMaxSharedB || a->n_groups > kMaxGroups) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

int check(const gdn_shared_attn_args* a) {
  int rc = check_sizes(a);
  if (rc == GDN_OK) rc = check(&a->attn);
  if (rc != GDN_OK || a->attn.B == 0 || a->attn.n_q_rows == 0) return rc;
  if (a->n_groups > 0 && (!a->group_start || !a->prefix_len)) return GDN_ERR_INVALID_ARG;
  if (a->lse && a->lse_row_stride < a->attn.H_q) return GDN_ERR_INVALID_ARG;
  auto al = [](const void* ptr) { return reinterpret_cast<uintptr_t>(ptr) % 4 == 0; };
  return al(a->group_start) && al(a->prefix_len) && al(a->lse) ? GDN_OK : GDN_ERR_MISALIGNED;
}

// The most rows that can take part in a prefix: prompts, whose rows fill tiles, do not, and need no places.
int64_t ranks(const gdn_paged_attn_args& a) {
  const int64_t most = most_rows(a.in_dtype == GDN_DTYPE_BF16 ? tc_rows() : kSimtRows, a.H_q / a.H_kv);
  return std::min((int64_t)a.n_q_rows, a.B * most);
}
// First parts of prefixes and of requests, one of each for a rank and head.  4096 requests of 127 rows and 2^31 heads of 256
// columns are below 2^62 bytes.
size_t places(const gdn_paged_attn_args& a) { return 2 * (size_t)ranks(a) * a.H_q; }

}  // namespace gdnattn

using namespace gdnattn;

// the attention's notes and partials, for every place its columns and its entry, and the ranked rows
extern "C" GDN_API size_t gdn_shared_attention_work_bytes(const gdn_shared_attn_args* args) {
  if (check_sizes(args) != GDN_OK) return 0;
  const size_t partials = gdn_paged_attention_work_bytes(&args->attn);
  return partials == 0 ? 0 : partials + places(args->attn) * (args->attn.d * sizeof(float) + sizeof(int4)) + (ranks(args->attn) + 1) * sizeof(int);
}

extern "C" GDN_API int gdn_shared_attention(const gdn_shared_attn_args* a, void* stream) {
  const int rc = check(a);
  if (rc != GDN_OK || a->attn.B == 0 || a->attn.n_q_rows == 0) return rc;
  Params p = params_of(&a->attn);
  SharedParams sp = {};
  sp.n_groups = a->n_groups;
  sp.key_align = 1;
  sp.group_start = a->group_start;
  sp.prefix_len = a->prefix_len;
  sp.lse = a->lse;
  sp.lse_row = a->lse_row_stride;
  const size_t attn_bytes = gdn_paged_attention_work_bytes(&a->attn);
  set_work(p, a->attn.in_dtype, a->attn.work);
  sp.n_ranks = (int)ranks(a->attn);
  sp.entries = reinterpret_cast<int4*>(static_cast<char*>(a->attn.work) + attn_bytes);
  sp.dense = reinterpret_cast<float*>(sp.entries + places(a->attn));
  sp.rank_row = reinterpret_cast<int*>(sp.dense + places(a->attn) * p.d);
  sp.count = sp.rank_row + sp.n_ranks;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return a->attn.in_dtype == GDN_DTYPE_BF16 ? run_shared_tc(p, sp, st) : run_simt<true>(p, sp, st);
}
