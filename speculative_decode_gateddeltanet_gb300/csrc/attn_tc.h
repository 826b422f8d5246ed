// The tensor-core attention's launch, for gdn_attn.cu.
#pragma once
#include <cuda_runtime.h>

namespace gdnattn {
struct Params;
int tc_blocks();  // blocks of its launch
int tc_rows();    // rows of its tiles
int run_tc(Params& p, cudaStream_t st);
}  // namespace gdnattn
