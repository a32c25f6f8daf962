// Column sums of partial rows: the last stage of the weight and bias gradients
// that blocks of rows have summed on their own.
#pragma once
#include "launch.cuh"
#include "vec.cuh"

namespace dit {

// out[c] = sum over p of partial[p][c], c < n, in the same order every time: 32
// columns a block, each in 32 strands of a loss-free sum (the rows may be many),
// joined as a tree.  Two sums of n columns a launch (blockIdx.y), each with an
// output that may be NULL.
struct ColumnSums {
  const float* partial;
  int64_t rows, pitch;  // floats between partial rows
  int n;
  int64_t second;       // floats from the first sum's columns to the second's
  float* out[2];
};
template <int UNUSED = 0>
__global__ void __launch_bounds__(1024) column_sums_kernel(const ColumnSums a) {
  __shared__ float strands[32][33];
  float* out = a.out[blockIdx.y];
  wait_previous();
  if (!out) return;
  const float* partial = a.partial + blockIdx.y * a.second;
  const int c = blockIdx.x * 32 + threadIdx.x;
  LongSum s;
  if (c < a.n) {
    int64_t p = threadIdx.y;
    for (; p + 96 < a.rows; p += 128) {
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = partial[(p + 32 * i) * a.pitch + c];
#pragma unroll
      for (int i = 0; i < 4; ++i) s.add(v[i]);
    }
    for (; p < a.rows; p += 32) s.add(partial[p * a.pitch + c]);
  }
  strands[threadIdx.y][threadIdx.x] = s.value();
  __syncthreads();
  float v = strands[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int col = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && col < a.n) out[col] = v;
}
inline cudaError_t column_sums(const ColumnSums& a, cudaStream_t s) {
  return launch_kernel(column_sums_kernel<0>, dim3((a.n + 31) / 32, a.out[1] ? 2 : 1), dim3(32, 32), 0, s, 1, true, a);
}

}  // namespace dit
