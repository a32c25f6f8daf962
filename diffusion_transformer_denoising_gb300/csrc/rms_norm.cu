// RMS norm with the residual's addition: the host's part (the kernels are in rms_norm.cuh).
#include "rms_norm.cuh"

namespace dit {

using namespace norm;

namespace {

cudaError_t by_type(int dtype, const Norm& p, int mode, int64_t blocks, cudaStream_t s) {
  if (dtype == DIT_DTYPE_F32) return by_mode<float>(p, mode, blocks, s);
  if (dtype == DIT_DTYPE_BF16) return by_mode<__nv_bfloat16>(p, mode, blocks, s);
  return by_mode<__half>(p, mode, blocks, s);
}

}  // namespace

int64_t rms_norm_workspace(const dit_rms_norm_args& a) {
  if (!a.dweight || a.batch * a.tokens == 0) return 0;
  int64_t most = 0;  // enough for rows of any alignment
  for (const Rows kind : {WHOLE_ROWS, ALIGNED_ROWS, ODD_ROWS}) {
    const int64_t n = blocks_of(a, true, kind);
    most = n > most ? n : most;
  }
  return most * a.channels * (int64_t)sizeof(float);
}

cudaError_t rms_norm_run(const dit_rms_norm_args& a, bool backward, float* workspace, cudaStream_t s) {
  const int64_t rows = a.batch * a.tokens;
  if (rows == 0) return a.dweight ? cudaMemsetAsync(a.dweight, 0, (size_t)a.channels * 4, s) : cudaSuccess;
  Norm p{};
  p.x = a.x, p.res = a.residual, p.dy = a.dy, p.total = a.total, p.out = a.out;
  const int esz = a.dtype == DIT_DTYPE_F32 ? 4 : 2;
  const int out_bytes = a.out_dtype == DIT_DTYPE_E4M3 ? 16 / esz : 16, out_esz = a.out_dtype == DIT_DTYPE_E4M3 ? 1 : esz;
  for (int i = 0; i < 2; ++i) {
    p.sx[i] = a.x_stride[i], p.sres[i] = a.residual_stride[i], p.stotal[i] = a.total_stride[i];
    p.sdy[i] = a.dy_stride[i], p.sout[i] = a.out_stride[i];
  }
  auto aligned = [&](const void* q, const int64_t (&st)[2], int e, int bytes) {
    return (((uintptr_t)q | (uintptr_t)(st[0] * e) | (uintptr_t)(st[1] * e)) & (bytes - 1)) == 0;
  };
  p.aligned = (aligned(p.x, p.sx, esz, 16) ? AL_X : 0) | (aligned(p.res, p.sres, esz, 16) ? AL_RES : 0) |
              (aligned(p.total, p.stotal, esz, 16) ? AL_TOTAL : 0) | (aligned(p.dy, p.sdy, esz, 16) ? AL_DY : 0) |
              (aligned(p.out, p.sout, out_esz, out_bytes) ? AL_OUT : 0) | (((uintptr_t)a.weight & 15) == 0 ? AL_W : 0);
  p.scale = a.scale, p.w = a.weight;
  p.rows = (uint32_t)rows, p.tokens = (uint32_t)a.tokens;
  p.C = a.channels, p.eps = a.eps;
  const Rows kind = rows_kind(p, 16 / esz);
  p.words = esz == 2 && (kind == ODD_ROWS || a.channels % 8) && aligned(p.x, p.sx, esz, 4) && aligned(p.res, p.sres, esz, 4) &&
            aligned(p.total, p.stotal, esz, 4) && aligned(p.dy, p.sdy, esz, 4) &&
            (a.out_dtype == DIT_DTYPE_E4M3 || aligned(p.out, p.sout, esz, 4));
  if (!backward) {
    const int64_t blocks = blocks_of(a, false, kind);
    return by_type(a.dtype, p, a.out_dtype == DIT_DTYPE_E4M3 ? E4M3 : SAME, blocks, s);
  }
  const int64_t blocks = blocks_of(a, true, kind);
  p.partial = a.dweight ? workspace : nullptr;
  const cudaError_t e = by_type(a.dtype, p, GRAD, blocks, s);
  if (e != cudaSuccess || !a.dweight) return e;
  return column_sums(ColumnSums{workspace, blocks, a.channels, a.channels, 0, {a.dweight, nullptr}, 0}, s);
}

}  // namespace dit
