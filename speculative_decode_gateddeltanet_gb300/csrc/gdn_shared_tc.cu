// gdn_shared_attention in bf16 on the tensor cores.
#include "attn_tc.cuh"

namespace gdnattn {

int run_shared_tc(const Params& p, const SharedParams& sp, cudaStream_t st) { return run<true>(p, sp, st); }

}  // namespace gdnattn
