// The tensor-core attention's launch, for gdn_attn.cu.
#pragma once
#include <cuda_runtime.h>

namespace gdnattn {
struct Params;
struct SharedParams;
int tc_blocks();  // blocks of its launch
int tc_rows();    // rows of its tiles
int run_tc(Params& p, cudaStream_t st);
int run_shared_tc(const Params& p, const SharedParams& sp, cudaStream_t st);
}  // namespace gdnattn
