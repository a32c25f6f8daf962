// Host-side TMA tensor-map construction (driver entry point fetched through
// the runtime, so the library does not link libcuda directly).
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace dit {

// Opt-in dynamic shared memory of a kernel, set once per device: the
// attribute belongs to the device's context, so a process that drives
// several GPUs sets it on each of them (on the current device).
constexpr int kMaxDevices = 64;
struct SmemAttr {
  int bytes[kMaxDevices] = {};
};
inline cudaError_t ensure_smem_attr(const void* func, int bytes, SmemAttr& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (done.bytes[dev] >= bytes) return cudaSuccess;
  e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.bytes[dev] = bytes;
  return e;
}

inline PFN_cuTensorMapEncodeTiled_v12000 tmap_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  return fn;
}

// The allocation that a device pointer lies in; false where the driver cannot say.
inline bool allocation_of(const void* p, uintptr_t* base, size_t* size) {
  static PFN_cuMemGetAddressRange_v3020 fn = nullptr;
  if (!fn) {
    cudaDriverEntryPointQueryResult q;
    void* f = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuMemGetAddressRange", &f, 3020, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return false;
    fn = reinterpret_cast<PFN_cuMemGetAddressRange_v3020>(f);
  }
  CUdeviceptr at = 0;
  if (fn(&at, size, (CUdeviceptr)(uintptr_t)p) != CUDA_SUCCESS) return false;
  *base = (uintptr_t)at;
  return true;
}

// Tensor of rank 2 or 3, dims innermost first, 128-byte swizzle unless told
// otherwise, out-of-bounds elements read as zero.  Returns false if the driver
// rejects it (base not 16-byte aligned, stride not a multiple of 16 bytes, a
// swizzled box row over 128 bytes, ...).
inline bool make_tmap(CUtensorMap* m, CUtensorMapDataType dt, const void* base, int rank, const uint64_t* dims,
                      const uint64_t* stride_bytes, const uint32_t* box,
                      CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  auto enc = tmap_encoder();
  if (!enc) return false;
  cuuint64_t d[3], st[2];
  cuuint32_t b[3], es[3] = {1, 1, 1};
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    b[i] = box[i];
  }
  for (int i = 0; i < rank - 1; ++i) st[i] = stride_bytes[i];
  CUresult r = enc(m, dt, rank, const_cast<void*>(base), d, st, b, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}
inline bool make_tmap_bf16(CUtensorMap* m, const void* base, int rank, const uint64_t* dims,
                           const uint64_t* stride_bytes, const uint32_t* box) {
  return make_tmap(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, rank, dims, stride_bytes, box);
}

}  // namespace dit
