// The RMS norm's kernels on bf16 activations.
#include "rms_norm.cuh"

template cudaError_t dit::norm::by_mode<__nv_bfloat16>(const dit::norm::Norm&, int, int64_t, cudaStream_t);
