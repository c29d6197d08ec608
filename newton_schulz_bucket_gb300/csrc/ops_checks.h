// What the layer operators' entry points share on the host: statuses with a
// message, sizes, and the check of the stream.
#pragma once

#include <cstdarg>
#include <cstdio>

#include <cuda_runtime.h>

#include "../../include/muon_ops.h"
#include "internal.h"
#include "ops.h"

namespace muon {

inline muon_status_t fail(muon_status_t st, const char* fmt, ...) {
  char buf[320];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  set_last_error(buf);
  return st;
}

inline muon_status_t cuda_status(const char* what, cudaError_t e) {
  return e == cudaSuccess ? MUON_OK : fail(MUON_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

inline bool dtype_ok(int32_t t) { return t == DT_F32 || t == DT_F16 || t == DT_BF16; }
inline int64_t dtype_size(int32_t t) { return t == DT_F32 ? 4 : 2; }

constexpr int64_t kMaxDim = 1ll << 30;
constexpr int64_t kMaxStride = 1ll << 36;
constexpr int64_t kMaxBlocks = 0x7fffffffll - 1024;  // (item counters run ahead by a grid's pairs)
inline size_t align256(size_t v) { return (v + 255) / 256 * 256; }

// Launches go to the current device, so the stream has to be one of its own.
// A capturing stream cannot be asked (the query would end the capture).
inline muon_status_t check_stream(const char* what, void* stream) {
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (s == nullptr || s == cudaStreamLegacy || s == cudaStreamPerThread) return MUON_OK;
  cudaStreamCaptureStatus capturing = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(s, &capturing) == cudaSuccess && capturing != cudaStreamCaptureStatusNone) return MUON_OK;
  int dev = 0, sdev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return fail(MUON_ERR_CUDA, "%s: cudaGetDevice failed", what);
  if (cudaStreamGetDevice(s, &sdev) != cudaSuccess) {
    cudaGetLastError();  // not left for the next call to report
    return fail(MUON_ERR_INVALID_ARG, "%s: stream is not a valid CUDA stream", what);
  }
  if (sdev != dev)
    return fail(MUON_ERR_INVALID_ARG, "%s: stream belongs to another device than the current one", what);
  return MUON_OK;
}

// A workspace argument that has to hold `need` bytes.
inline muon_status_t check_workspace(const char* what, const void* workspace, size_t bytes, size_t need) {
  if (need > 0 && (!workspace || bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255) != 0))
    return fail(MUON_ERR_INVALID_ARG, "%s: needs a 256-byte aligned workspace of %zu bytes", what, need);
  return MUON_OK;
}

}  // namespace muon
