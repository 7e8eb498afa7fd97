// Host-side pieces shared by the entry points in gqa_api.cu and block_api.cu:
// the handle, the per-thread error text and small tensor checks.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <vector>

#include "../../include/gqa.h"

struct gqa_handle {
  gqa_attrs attrs;
  long long wait_budget;    // bound of each pipeline wait of the tensor-core kernels (clock cycles)
  int withhold_tile;        // >= 0: testing the timeout path (see gqa_set_wait_limit)
  // per-launch profiling (gqa_profile_begin / gqa_profile_end)
  bool profiling;
  std::vector<cudaEvent_t> events;  // 2 per launch
  std::vector<int> kinds;
  int used;
};

namespace gqa {

// Records the reason of a failure for gqa_last_error (this thread) and returns `s`.
gqa_status fail(gqa_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

inline gqa_status cuda_fail(cudaError_t e, const char* what) {
  return fail(GQA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

constexpr size_t kAlign = 256;
inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

inline bool present(const gqa_tensor& t) { return t.data != nullptr; }

inline bool shape_is(const gqa_tensor& t, int ndim, const int64_t* s) {
  if (t.ndim != ndim) return false;
  for (int i = 0; i < ndim; ++i)
    if (t.shape[i] != s[i]) return false;
  return true;
}

inline gqa_status check_aligned(const gqa_tensor& t, const char* name) {
  if (present(t) && (reinterpret_cast<uintptr_t>(t.data) & 15u) != 0)
    return fail(GQA_ERR_INVALID_ARGUMENT, "%s: data pointer is not 16-byte aligned", name);
  return GQA_OK;
}

// Launch through `fn`, bracketed by an event pair when the handle is profiling.
template <typename F>
cudaError_t timed_launch(gqa_handle* h, int kind, cudaStream_t st, F fn) {
  const bool rec = h->profiling && h->used < (int)h->kinds.size();
  if (rec) cudaEventRecord(h->events[2 * h->used], st);
  cudaError_t e = fn();
  if (rec) {
    cudaEventRecord(h->events[2 * h->used + 1], st);
    h->kinds[h->used++] = kind;
  }
  return e;
}

}  // namespace gqa
