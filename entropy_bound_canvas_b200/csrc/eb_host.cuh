// eb_host.cuh -- host helpers shared by the library's C entry points: the
// current device's guard, workspace layout and tensor maps.
#pragma once

#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstddef>
#include <cstdint>
#include <cstring>
#include <mutex>

namespace ebk {

// Makes a device current, and the caller's again on scope exit.
struct DeviceGuard {
  int prev = -1;  // to restore; -1: it was current already
  bool ok = false;
  explicit DeviceGuard(int dev) {
    int now = -1;
    if (cudaGetDevice(&now) != cudaSuccess) return;
    if (now == dev) {
      ok = true;
      return;
    }
    if (cudaSetDevice(dev) == cudaSuccess) {
      prev = now;
      ok = true;
    }
  }
  ~DeviceGuard() {
    if (prev >= 0) cudaSetDevice(prev);
  }
};

inline size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// Zeros device memory of the current device before it returns, whatever the
// device's other streams hold.  (cudaMemset on device memory returns early, on
// a stream that non-blocking streams do not wait for: a handle's first call
// could be under way when its workspace is cleared.)
inline bool clear_now(void* p, size_t bytes) {
  cudaStream_t st = nullptr;
  bool ok = cudaStreamCreateWithFlags(&st, cudaStreamNonBlocking) == cudaSuccess;
  if (ok) {
    ok = cudaMemsetAsync(p, 0, bytes, st) == cudaSuccess;
    ok = cudaStreamSynchronize(st) == cudaSuccess && ok;
    ok = cudaStreamDestroy(st) == cudaSuccess && ok;
  }
  if (!ok) cudaGetLastError();
  return ok;
}

// A kernel launched as a programmatic dependent of the previous one on `st`.
inline bool launch_dependent(const void* fn, dim3 grid, dim3 block, size_t smem, void** args,
                             cudaStream_t st) {
  cudaLaunchConfig_t lc;
  std::memset(&lc, 0, sizeof(lc));
  lc.gridDim = grid;
  lc.blockDim = block;
  lc.dynamicSmemBytes = smem;
  lc.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return cudaLaunchKernelExC(&lc, fn, args) == cudaSuccess;
}

inline PFN_cuTensorMapEncodeTiled_v12000 tmap_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    cudaGetLastError();
  });
  return fn;
}

// A bf16 matrix [outer][inner] (inner contiguous), read in boxes of
// box_outer x box_inner with the 128-byte swizzle the MMA descriptors expect.
inline bool make_tmap(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer,
                      uint32_t box_inner, uint32_t box_outer) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tmap_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {inner * 2};
  cuuint32_t box[2] = {box_inner, box_outer};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

}  // namespace ebk
