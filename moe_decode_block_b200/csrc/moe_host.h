// moe_host.h -- host helpers shared by the library's translation units.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "moe_decode.h"

namespace moe {

// Record a CUDA error for moe_decode_last_cuda_error; returns MOE_ERR_CUDA.
int host_fail_cuda(cudaError_t e);

// Set device memory to zero before returning.  (cudaMemset returns early, and
// its stream, the legacy default one, is not waited for by streams made with
// cudaStreamNonBlocking, as torch's are: behind other work it could come after
// kernels that need the zeros, or under them.)
inline cudaError_t host_zero_now(void* p, size_t bytes) {
  cudaStream_t st = nullptr;
  cudaError_t e = cudaStreamCreateWithFlags(&st, cudaStreamNonBlocking);
  if (e != cudaSuccess) return e;
  e = cudaMemsetAsync(p, 0, bytes, st);
  const cudaError_t s = cudaStreamSynchronize(st);
  cudaStreamDestroy(st);
  return e != cudaSuccess ? e : s;
}

inline bool host_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int kHostMaxDevices = 64;

// The current device, checked once per device to be compute capability 10.x.
// MOE_OK and *dev, *num_sms, or an error code.
int host_current_device(int* dev, int* num_sms);

// Raise a kernel's dynamic shared-memory limit on the current device, once
// per kernel and device (`done` belongs to the kernel).
template <typename K>
int host_raise_smem(K kern, int bytes, int dev, std::atomic<uint64_t>& done) {
  const uint64_t bit = 1ull << dev;
  if (done.load(std::memory_order_acquire) & bit) return MOE_OK;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return host_fail_cuda(e);
  done.fetch_or(bit, std::memory_order_release);
  return MOE_OK;
}

// Whether the next launch of a tcgen05 4-bit kernel holds its first step back
// (moe_w4_test_hold); counts it.
int host_w4_hold();

// Launch with an optional cluster size and programmatic dependent launch.
template <typename... KArgs, typename... Args>
cudaError_t host_launch(void (*kern)(KArgs...), dim3 grid, int block, size_t smem, cudaStream_t st, int cluster,
                        bool pdl, Args&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = (unsigned)cluster;
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = n ? attr : nullptr;
  cfg.numAttrs = (unsigned)n;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

}  // namespace moe
