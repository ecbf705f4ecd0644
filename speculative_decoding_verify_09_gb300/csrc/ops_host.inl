// What the operators' files share: the thread-local error text behind
// sv_last_error() (api.cu), and how their kernels are launched.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "spec_ops.h"

namespace sv {

// Records the message of a failed call and returns its status.
sv_status record_error(sv_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));

// The checks of spec_rope_rows (rope.cu), in the name of entry point `who`.
sv_status check_rope(const sv_rope_args *a, const char *who);

// SMs of the current device (0 if it cannot be asked).
int device_sms();

// Launches a kernel whose launch is worked on while the kernel before it on the
// stream still runs (programmatic dependent launch): between small kernels on a
// stream that saves up to 3 us each (calls from a host loop without and with it: bass_b8
// verify rows adjusted 8.2 and 6.6 us, 176 rotary rows 6.1 and 4.1, 64 prompts counted
// 10.2 and 7.4; between a graph's nodes 0.2 to 0.6 us).  Such a kernel begins with
// wait_for_previous(), before it touches global memory, and reads by ordinary loads
// (or from L2): it may be resident while the kernel before still writes, and the
// read-only path (__ldg) is only for data that nobody writes while it runs.  None of
// them lets its successor start before it is done, which would put waiting CTAs
// on its SMs.
template <typename Params>
inline cudaError_t launch_behind(void (*kernel)(Params), dim3 grid, int threads, size_t smem,
                                 cudaStream_t s, const Params &params) {
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, params);
  if (e != cudaSuccess) cudaGetLastError();     // reported by the caller, not left for another call
  return e;
}

// The most dynamic shared memory that calls of one kernel take.  What the driver allows a kernel is
// raised to it once per device, and never set to what one call needs: that would be the limit of
// another host thread's launch, too.
struct SharedLimit {
  const size_t most;
  std::atomic<uint64_t> ready{0};                   // a bit per device
  explicit SharedLimit(size_t bytes) : most(bytes) {}
  cudaError_t raise(const void *kernel) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t{1} << (dev & 63);
    if (dev < 64 && (ready.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
    if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_release);
    return e;
  }
};

// launch_behind for a kernel whose calls may take more dynamic shared memory than the default allows.
template <typename Params>
inline cudaError_t launch_after_previous(void (*kernel)(Params), SharedLimit &limit, dim3 grid, int threads,
                                         size_t smem, cudaStream_t s, const Params &params) {
  if (smem > limit.most) return cudaErrorInvalidValue;
  if (limit.most > 48 * 1024) {
    const cudaError_t e = limit.raise(reinterpret_cast<const void *>(kernel));
    if (e != cudaSuccess) {
      cudaGetLastError();
      return e;
    }
  }
  return launch_behind(kernel, grid, threads, smem, s, params);
}

// Waits until the kernel before has completed and its writes are visible.
__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
}

inline bool is_aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace sv
