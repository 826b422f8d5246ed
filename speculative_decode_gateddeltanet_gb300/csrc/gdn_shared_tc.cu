// gdn_shared_attention in bf16 on the tensor cores.
#include "attn_tc.cuh"

namespace gdnattn {

int run_shared_tc(const Params& p, const SharedParams& sp, cudaStream_t st) { return run<true>(p, sp, st); }

}  // namespace gdnattn

#ifdef GDN_TEST_HOOKS
// Test builds only: drop the first K copy of block `block` of later calls (-1 restores it).
extern "C" GDN_API int gdn_test_drop_shared_copy(int block) {
  return cudaMemcpyToSymbol(gdnattn::g_test_drop_block, &block, sizeof(int)) == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}
#endif
