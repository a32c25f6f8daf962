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

int64_t rms_norm_workspace(const dit_rms_norm_args& a);
cudaError_t rms_norm_run(const dit_rms_norm_args& a, bool backward, float* workspace, cudaStream_t s);

int64_t gated_ffn_workspace(const dit_gated_ffn_args& a, bool backward);
cudaError_t gated_ffn_run(const dit_gated_ffn_args& a, bool backward, void* workspace, cudaStream_t s);
// Waits for the stream, then takes the site of a wait that ran out (0: none).
cudaError_t gated_ffn_take_error(int* site, cudaStream_t s);

int64_t grad_norm_workspace(const dit_grad_tensor* t, int64_t n);
cudaError_t grad_norm_run(const dit_grad_tensor* t, int64_t n, float max_norm, float* norm, void* workspace,
                          cudaStream_t s);

}  // namespace dit
