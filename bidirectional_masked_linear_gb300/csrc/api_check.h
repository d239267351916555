// api_check.h -- what the entry points of the token-major operators share (no
// device code): checks of pointers, types and strides, and the workspace.
#pragma once

#include <stdint.h>

#include "../../include/lion.h"
#include "ssm_check.h"

namespace lion {
namespace api {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Checks of a call's pointers: aligned to `a` bytes and memory that the current device's kernels can use.
class Pointers {
 public:
  Pointers() {
    if (cudaGetDevice(&device_) != cudaSuccess) cudaGetLastError();   // no device: no pointer passes
  }
  bool need(const void* p, size_t a) const { return p && aligned(p, a) && usable(p); }
  bool maybe(const void* p, size_t a) const { return !p || need(p, a); }

 private:
  bool usable(const void* p) const {
    cudaPointerAttributes at;
    if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
      cudaGetLastError();
      return false;
    }
    return lion::usable_on(at, device_);
  }
  int device_ = -1;
};

inline bool dtype_ok(int t) { return t == LION_DTYPE_BF16 || t == LION_DTYPE_FP32; }
inline size_t esize(int t) { return t == LION_DTYPE_BF16 ? 2 : 4; }
inline bool flag(int v) { return v == 0 || v == 1; }
inline bool stride_ok(long long ld, long long width) { return ld == 0 || ld >= width; }

constexpr long long kMaxGrid = 0x7fffffffLL;

inline lion_status from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return LION_OK;
  if (e == cudaErrorMemoryAllocation) return LION_ERR_NO_MEMORY;
  return LION_ERR_CUDA;
}

// Runs `go(workspace)` on the caller's workspace or on a stream-ordered one.
template <typename F>
lion_status with_workspace(void* ws, size_t ws_bytes, size_t want, cudaStream_t s, F go) {
  if (want == 0) return from_cuda(go(nullptr));
  if (ws) {
    if (!Pointers().need(ws, 256) || ws_bytes < want) return LION_ERR_INVALID_ARG;
    return from_cuda(go(ws));
  }
  cudaError_t e = cudaMallocAsync(&ws, want, s);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return from_cuda(e);
  }
  e = go(ws);
  const cudaError_t f = cudaFreeAsync(ws, s);
  return from_cuda(e != cudaSuccess ? e : f);
}

}  // namespace api
}  // namespace lion
