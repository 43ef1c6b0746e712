// vx_api.h -- what the translation units with C entry points share: argument
// checks, the launch context of a call and the carving of its workspace.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "vx.h"
#include "vx_internal.h"

namespace vx {

constexpr size_t kStatusBytes = 256;
constexpr size_t kAlign = 1024;

inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Bump allocator over the caller's workspace (or a size counter when base is null).
struct Carve {
  uint8_t* base;
  size_t off;
  void* take(size_t bytes) {
    off = align_up(off, kAlign);
    void* p = base ? base + off : nullptr;
    off += bytes;
    return p;
  }
};

#define VX_CHECK_ARG(cond, ...)   \
  do {                            \
    if (!(cond)) {                \
      set_error(__VA_ARGS__);     \
      return VX_ERR_INVALID_ARG;  \
    }                             \
  } while (0)

#define VX_CUDA(call)                                                          \
  do {                                                                         \
    cudaError_t e_ = (call);                                                   \
    if (e_ != cudaSuccess) {                                                   \
      set_error("%s failed: %s", #call, cudaGetErrorString(e_));               \
      return VX_ERR_CUDA;                                                      \
    }                                                                          \
  } while (0)

inline vx_status make_launch(Launch* L, void* ws, size_t ws_bytes, size_t need, cudaStream_t stream) {
  VX_CHECK_ARG(ws != nullptr, "workspace is null");
  VX_CHECK_ARG((reinterpret_cast<uintptr_t>(ws) & 255) == 0, "workspace must be 256-byte aligned");
  VX_CHECK_ARG(ws_bytes >= need, "workspace too small: %zu bytes given, %zu needed", ws_bytes, need);
  L->stream = stream;
  L->status = static_cast<DevStatus*>(ws);
  L->limit_ns = wait_limit_ns();
  L->sm_count = current_sm_count();
  if (L->sm_count <= 0) {
    set_error("no CUDA device is current");
    return VX_ERR_CUDA;
  }
  return VX_OK;
}

}  // namespace vx
