// Column sums of partial rows: the last stage of the weight and bias gradients
// that blocks of rows have summed on their own.
#pragma once
#include "launch.cuh"
#include "vec.cuh"

namespace dit {

// out[c] = sum over p of partial[p][c], c < n, in the same order every time: 8 columns
// a block, each in 64 strands of a loss-free sum (the rows may be many), joined as a
// tree.  Two sums of n columns a launch (blockIdx.y), each with an output that may be NULL.
struct ColumnSums {
  const float* partial;
  int64_t rows, pitch;  // floats between partial rows
  int n;
  int64_t second;       // floats from the first sum's columns to the second's
  float* out[2];
  int late;             // the kernels before the previous one have written what is read (launch.cuh)
};
constexpr int kSumColumns = 8, kSumStrands = 64;
template <int UNUSED = 0>
__global__ void __launch_bounds__(kSumColumns * kSumStrands) column_sums_kernel(const ColumnSums a) {
  __shared__ float strands[kSumColumns][kSumStrands + 1];
  float* out = a.out[blockIdx.y];
  const int col = threadIdx.x % kSumColumns, strand = threadIdx.x / kSumColumns;
  const int c = blockIdx.x * kSumColumns + col;
  if (!a.late) wait_previous();
  start_next();
  LongSum s;
  if (out && c < a.n) {
    const float* p = a.partial + blockIdx.y * a.second + c;
    constexpr int U = 8;  // loads under way
    for (int64_t r = strand; r < a.rows; r += U * kSumStrands) {
      float v[U];
#pragma unroll
      for (int i = 0; i < U; ++i) v[i] = r + i * kSumStrands < a.rows ? __ldcg(p + (r + i * kSumStrands) * a.pitch) : 0.f;
#pragma unroll
      for (int i = 0; i < U; ++i) s.add(v[i]);
    }
  }
  strands[col][strand] = s.value();
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (out && warp < kSumColumns) {
    float v = strands[warp][lane] + strands[warp][lane + 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0 && blockIdx.x * kSumColumns + warp < a.n) out[blockIdx.x * kSumColumns + warp] = v;
  }
  if (a.late) wait_previous();  // the call's end is the end of all its kernels
}
inline cudaError_t column_sums(const ColumnSums& a, cudaStream_t s) {
  return launch_kernel(column_sums_kernel<0>, dim3((a.n + kSumColumns - 1) / kSumColumns, a.out[1] ? 2 : 1),
                       dim3(kSumColumns * kSumStrands), 0, s, 1, true, a);
}

}  // namespace dit
