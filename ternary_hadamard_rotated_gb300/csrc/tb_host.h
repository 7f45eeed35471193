// Host-side helpers of the C ABI: argument checks, CUDA error capture, device facts.
#pragma once

#include <cudaTypedefs.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/tb.h"

namespace tb {

// remember the text of a CUDA error for tb_last_cuda_error()
void record_cuda_error(cudaError_t e);

inline int check_launch() {
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return TB_ERR_CUDA;
  }
  return TB_OK;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Hadamard block sizes the transform accepts (the pack's loader takes 512 .. 4096); 1024 is the
// pack's own and the one the fused kernels run, the others go through a separate transform
inline bool supported_block(int block) {
  return block == 512 || block == 1024 || block == 2048 || block == 4096;
}

inline bool aligned_to(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// tokens per page of the K/V cache: a power of two, 16 .. 256
inline bool supported_page(int64_t page) {
  return page == 16 || page == 32 || page == 64 || page == 128 || page == 256;
}
inline int log2_of(int64_t p) {
  int n = 0;
  while ((1ll << n) < p) ++n;
  return n;
}

// head widths of the attention kernels
inline bool supported_head(int64_t D) { return D == 64 || D == 128 || D == 256; }

// y = fwht(x) over blocks of `block` (a supported size; K a multiple of it); y may equal x
int launch_fwht(const __half* x, __half* y, const int8_t* signs, int64_t M, int64_t K, int block,
                int inverse, cudaStream_t s);

// cuTensorMapEncodeTiled, looked up once (thread-safe); null when the driver lacks it
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// streaming multiprocessors and opt-in shared memory of the current device
struct DeviceFacts {
  int device = -1;
  int sms = 0;
  int smem_optin = 0;
};
int device_facts(DeviceFacts* f);

// cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes), made only when
// bytes exceeds what was set before for this kernel on this device (a driver call per launch
// costs host time that a stream of small launches does not hide)
int ensure_dynamic_smem(const void* func, int device, int bytes);

}  // namespace tb
