// Host-side helpers shared by the C-ABI translation units: status codes,
// the thread-local last-error message and CUDA error mapping.
#pragma once

#include <atomic>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <exception>
#include <string>

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include "pka.h"

namespace pka {

// Records `fmt` as the calling thread's last error and returns `code`.
int fail(int code, const char* fmt, ...);

// Clears the calling thread's last error.
void clear_error();

// Maps a CUDA runtime error to PKA_ERR_CUDA with a message naming `what`.
// Raises a kernel's dynamic shared memory limit once per device: `done` is the
// calling launcher's own bit set (devices 0-63; a higher device sets it on
// every launch).  The attribute stays set for the life of the process.  carveout: an SM that
// runs the kernel gives shared memory all that it can, so that other kernels' CTAs fit beside.
template <typename Kernel>
inline cudaError_t set_smem_once(Kernel kern, int bytes, std::atomic<uint64_t>& done, bool carveout = false) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
  if (bit != 0 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && carveout)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess && bit != 0) done.fetch_or(bit, std::memory_order_acq_rel);
  return e;
}

inline int cuda_fail(cudaError_t e, const char* what) {
  (void)cudaGetLastError();   // reported here: not again at the next launch
  return fail(PKA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// For waits and releases that nothing depends on: what CUDA refuses there (it does while a
// stream of this thread captures) is not found by the next launch either.
inline void ignored(cudaError_t e) {
  if (e != cudaSuccess) (void)cudaGetLastError();
}

inline bool aligned(const void* p, uintptr_t n) {
  return (reinterpret_cast<uintptr_t>(p) % n) == 0;
}

inline size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// An NVTX range over an entry point, so that the plan and run calls show up by
// name on a profiler's timeline (a no-op call when no tool is attached).
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

// PKA_OK when `plan_device` is the current device.
int check_device(int plan_device);

// Waits for `stream`, reads and clears a device status word, and maps its bits
// to an error code.
int read_status(int32_t* d_status, cudaStream_t stream);

// Runs `f`, turning a C++ exception (a host allocation that failed) into an error code.
template <typename F>
int guarded(F&& f) {
  try {
    return f();
  } catch (const std::exception& e) {
    return fail(PKA_ERR_INVALID_ARG, "host error: %s", e.what());
  }
}

// A byte range, and whether two share a byte.
struct Range {
  const void* p;
  size_t n;
};
inline bool overlap(const Range& x, const Range& y) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
  return x.n > 0 && y.n > 0 && a < b + y.n && b < a + x.n;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace pka

#define PKA_CHECK_ARG(cond, ...)                          \
  do {                                                    \
    if (!(cond)) return ::pka::fail(PKA_ERR_INVALID_ARG, __VA_ARGS__); \
  } while (0)

#define PKA_CUDA_TRY(expr, what)                          \
  do {                                                    \
    cudaError_t _e = (expr);                              \
    if (_e != cudaSuccess) return ::pka::cuda_fail(_e, what); \
  } while (0)
