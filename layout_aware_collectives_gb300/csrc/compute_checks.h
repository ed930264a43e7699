// Argument checks and the handle's device binding, which the C entries of the
// feed-forward unit (compute_api.cpp) and of the expert layer (expert_api.cpp)
// share.
#pragma once

#include <string>

#include "compute_internal.h"

#define TIDE_TRY(call)                  \
  do {                                  \
    const tide_status_t s_ = (call);    \
    if (s_ != TIDE_OK) return s_;       \
  } while (0)

// No exception (of a message's or a lock's making) leaves a C entry.
#define TIDE_CATCH \
  catch (...) { return TIDE_ERR_OUT_OF_MEMORY; }

namespace tide {

constexpr int64_t kMaxDim = INT32_MAX;
constexpr int64_t kMaxNumel = (int64_t)1 << 38;

inline tide_status_t invalid(const std::string& msg) { return set_error(TIDE_ERR_INVALID_ARG, msg); }

inline tide_status_t check_dims(int64_t a, int64_t b, const char* what) {
  if (a < 0 || b < 0 || a > kMaxDim || b > kMaxDim || (b && a > kMaxNumel / b))
    return invalid(std::string(what) + ": sizes out of range");
  return TIDE_OK;
}

inline tide_status_t check_buffer(const void* p, int64_t numel, const char* what) {
  if (numel == 0) return TIDE_OK;
  if (!p) return invalid(std::string(what) + " is NULL");
  if ((uintptr_t)p & 15u) return set_error(TIDE_ERR_MISALIGNED, std::string(what) + " is not 16-byte aligned");
  return TIDE_OK;
}

// A matrix of `rows` rows of `cols` elements, `ld` apart.
inline tide_status_t check_matrix(const void* p, int64_t rows, int64_t cols, int64_t ld, const char* what) {
  TIDE_TRY(check_buffer(p, rows * cols, what));
  if (ld < cols || (rows && ld > kMaxNumel / rows)) return invalid(std::string(what) + ": row stride out of range");
  return TIDE_OK;
}

inline tide_status_t check_blocks(const void* codes, const void* scales, int64_t rows, int64_t cols, const char* what) {
  TIDE_TRY(check_buffer(codes, rows * cols, (std::string(what) + " codes").c_str()));
  if (rows * cols == 0) return TIDE_OK;
  if (!scales) return invalid(std::string(what) + " scales is NULL");
  if ((uintptr_t)scales & 3u) return set_error(TIDE_ERR_MISALIGNED, std::string(what) + " scales is not 4-byte aligned");
  return TIDE_OK;
}

inline bool capturing(cudaStream_t stream) {
  cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(stream, &st) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  return st == cudaStreamCaptureStatusActive;
}

// The current device, which is a bound handle's.
inline tide_status_t current_device(const tide_compute_s* c, int* dev) {
  const cudaError_t e = cudaGetDevice(dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (c->device >= 0 && *dev != c->device)
    return invalid("handle is bound to device " + std::to_string(c->device) + " but device " + std::to_string(*dev) +
                   " is current");
  return TIDE_OK;
}

// Binds the handle to the current device on first use (compute_api.cpp).
tide_status_t bind(tide_compute_s* c, cudaStream_t stream);

inline TcLaunch launch_of(tide_compute_s* c) {
  std::lock_guard<std::mutex> g(c->mu);
  return TcLaunch{&c->dev, c->d_err, (uint64_t)c->test_stall_ns, (uint64_t)c->test_late_ns};
}

inline tide_status_t launched(cudaError_t e, const char* what) { return e == cudaSuccess ? TIDE_OK : cuda_fail(e, what); }

inline int64_t round256(int64_t v) { return (v + 255) / 256 * 256; }

}  // namespace tide
