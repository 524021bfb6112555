// tq_host.cuh -- host helpers shared by the library's translation units:
// error state, device check, alignment test and the launch wrapper.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/tq.h"

namespace tq_host {

inline thread_local int g_last_cuda_error = 0;

inline int cuda_fail(cudaError_t e) {
  g_last_cuda_error = (int)e;
  return TQ_ERR_CUDA;
}

#define TQ_CUDA(call)                           \
  do {                                          \
    cudaError_t e_ = (call);                    \
    if (e_ != cudaSuccess) return cuda_fail(e_); \
  } while (0)

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int kMaxDevices = 64;
inline int g_arch_ok[kMaxDevices];  // 0 unknown, 1 ok, 2 bad
inline int g_num_sms[kMaxDevices];

// Current device must be compute capability 10.0 (B200, sm_100a).
inline int check_arch(int* num_sms) {
  int dev = 0;
  TQ_CUDA(cudaGetDevice(&dev));
  if (dev < 0 || dev >= kMaxDevices) return TQ_ERR_ARCH;
  if (g_arch_ok[dev] == 0) {
    int major = 0, minor = 0, sms = 0;
    TQ_CUDA(cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev));
    TQ_CUDA(cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev));
    TQ_CUDA(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
    g_num_sms[dev] = sms;
    g_arch_ok[dev] = (major == 10 && minor == 0) ? 1 : 2;
  }
  if (g_arch_ok[dev] != 1) return TQ_ERR_ARCH;
  if (num_sms) *num_sms = g_num_sms[dev];
  return TQ_OK;
}

// Launch with the programmatic-stream-serialization attribute so that a
// kernel may start its weight prefetch while the previous one finishes.
template <typename... KArgs, typename... Args>
int launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
#ifdef TQ_NO_PDL
  cfg.numAttrs = 0;  // build option: plain stream ordering
#else
  cfg.numAttrs = 1;
#endif
  TQ_CUDA(cudaLaunchKernelEx(&cfg, kernel, args...));
  return TQ_OK;
}

// Every workspace starts with a fixed region of per-tile arrival counters
// (kCounterBytes, so every call, whatever its shape, finds its counters in
// the same zeroed bytes; each call leaves them zero).  Everything after it
// (partial sums, activation scratch) is written before it is read.
constexpr size_t kCounterBytes = 64 * 1024;

}  // namespace tq_host
