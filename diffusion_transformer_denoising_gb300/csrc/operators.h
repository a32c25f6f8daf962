// Internal interface between the C ABI of the operators (operators_api.cu,
// which checks the arguments) and their kernels.  Nothing here is exported.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/dit.h"

namespace dit {

// dweight partials of the rotation's gradient: at most this many rows of
// head_dim floats (each of the two tensors launches at most half of them).
constexpr int kRopeGradBlocks = 1024;
// Whether the gradient joins its weight sums without them.
bool rope_one_cluster(const dit_rope_args& a);
cudaError_t rope_run(const dit_rope_args& a, bool backward, float* workspace, cudaStream_t s);

int64_t group_norm_workspace(const dit_group_norm_args& a, bool backward);
cudaError_t group_norm_run(const dit_group_norm_args& a, bool backward, float* workspace, cudaStream_t s);

}  // namespace dit
