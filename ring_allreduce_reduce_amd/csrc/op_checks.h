// What the block operators' entries share: refusals, checks of operands and
// workspaces (defined in block_ops.cpp).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <initializer_list>
#include <mutex>
#include <string>

#include "op_host.h"
#include "ringar.h"

namespace ringar {

ringar_result_t hip_fail(hipError_t e, const char* what);
ringar_result_t refuse(ringar_result_t code, const std::string& why);

#define HIP_TRY(call)                                   \
  do {                                                  \
    hipError_t e_ = (call);                             \
    if (e_ != hipSuccess) return hip_fail(e_, #call);   \
  } while (0)

#define TRY(call)                                       \
  do {                                                  \
    ringar_result_t r_ = (call);                        \
    if (r_ != RINGAR_SUCCESS) return r_;                \
  } while (0)

// ------------------------------------------------------------- workspaces
// The stream's workspace: `bytes` at *out (null where none are needed).  It
// starts with kCounters zeroed words, which every kernel that uses one leaves
// at zero; *out is what follows them.  The caller holds g_ws_mu from here to
// its last launch, so two threads on one stream cannot interleave.
extern std::mutex g_ws_mu;
constexpr int kCounters = 4096;
constexpr size_t kCounterBytes = kCounters * sizeof(uint32_t);
ringar_result_t workspace(hipStream_t st, size_t bytes, char** out);

// Parts of one workspace, each 256-byte aligned.
struct Layout {
  size_t bytes = 0;
  size_t add(size_t n) {
    const size_t at = bytes;
    bytes += (n + 255) / 256 * 256;
    return at;
  }
};

// ---------------------------------------------------------------- checks
inline size_t size_of(int dtype) { return dtype == RINGAR_FLOAT32 ? 4 : 2; }
inline bool type_ok(int dtype) { return dtype == RINGAR_FLOAT16 || dtype == RINGAR_BFLOAT16 || dtype == RINGAR_FLOAT32; }
constexpr int64_t kMaxPitch = 0x7fffffff;
constexpr int64_t kMaxDim = kMaxPitch - 1024;   // sizes rounded up to tiles stay 32-bit

inline bool dims_ok(std::initializer_list<int64_t> d) {
  for (int64_t v : d)
    if (v < 0 || v > kMaxDim) return false;
  return true;
}

// A matrix operand: rows x cols elements, row i at p + i * ld elements.
struct Mat {
  const char* name;
  const void* p;
  int64_t rows, cols, ld;
  size_t es;
  bool output;
  bool in_place = false;    // an input that may be y's very place
  bool any_place = false;   // an input that may be any output's
};

ringar_result_t check_mats(std::initializer_list<Mat> all);

#define VEC(name, p, n, es, out) Mat{name, p, (p) ? 1 : 0, n, n, es, out}

// No C++ exception leaves a C entry (allocation of a map node or a text).
template <typename F> ringar_result_t guarded(F f) {
  try {
    return f();
  } catch (...) {
    return RINGAR_ERR_INTERNAL;
  }
}

}  // namespace ringar
