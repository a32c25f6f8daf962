// The RMS norm's kernels on f32 activations.
#include "rms_norm.cuh"

template cudaError_t dit::norm::by_mode<float>(const dit::norm::Norm&, int, int64_t, cudaStream_t);
