// Argument checks shared by the entry points in block_api.cu and tree_api.cu.
#pragma once

#include "gqa_host.h"

namespace gqa {

inline size_t dtype_size(int32_t d) {
  switch (d) {
    case GQA_F32:
    case GQA_I32: return 4;
    case GQA_F16:
    case GQA_BF16: return 2;
    case GQA_I8:
    case GQA_U8: return 1;
  }
  return 0;
}

inline size_t bytes_of(const gqa_tensor& t) {
  size_t n = dtype_size(t.dtype);
  for (int i = 0; i < t.ndim; ++i) n *= (size_t)t.shape[i];
  return n;
}

inline bool overlap(const gqa_tensor& a, const gqa_tensor& b) {
  if (!present(a) || !present(b)) return false;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.data), pb = reinterpret_cast<uintptr_t>(b.data);
  return pa < pb + bytes_of(b) && pb < pa + bytes_of(a);
}

struct Named {
  const gqa_tensor* t;
  const char* name;
};

// Alignment of every tensor, and that no written one overlaps another (`same`
// pairs may be one buffer).
inline gqa_status check_buffers(const Named* read, int nread, const Named* written, int nwritten, const gqa_tensor* same[][2],
                         int nsame) {
  for (int k = 0; k < nread + nwritten; ++k) {
    const Named& n = k < nread ? read[k] : written[k - nread];
    gqa_status s = check_aligned(*n.t, n.name);
    if (s != GQA_OK) return s;
  }
  for (int i = 0; i < nwritten; ++i) {
    for (int k = 0; k < nread + i; ++k) {
      const Named& n = k < nread ? read[k] : written[k - nread];
      if (!overlap(*written[i].t, *n.t)) continue;
      bool ok = false;
      for (int x = 0; x < nsame; ++x)
        ok |= same[x][0] == written[i].t && same[x][1] == n.t && written[i].t->data == n.t->data;
      if (!ok) return fail(GQA_ERR_INVALID_ARGUMENT, "%s overlaps %s", written[i].name, n.name);
    }
  }
  return GQA_OK;
}

inline gqa_status check_float(const gqa_tensor& t, const char* name) {
  if (t.dtype == GQA_BF16) return fail(GQA_ERR_UNSUPPORTED, "bfloat16 is not implemented");
  if (t.dtype != GQA_F32 && t.dtype != GQA_F16)
    return fail(GQA_ERR_INVALID_ARGUMENT, "%s dtype must be float32 or float16", name);
  return GQA_OK;
}

inline gqa_status check_head_size(long long H) {
  if (H % 16 != 0 || H < 16 || H > 256)
    return fail(GQA_ERR_UNSUPPORTED, "head_size %lld: supported head sizes are multiples of 16 in [16, 256]", H);
  return GQA_OK;
}

inline gqa_status check_status_word(const void* status) {
  if (reinterpret_cast<uintptr_t>(status) & 3u)
    return fail(GQA_ERR_INVALID_ARGUMENT, "status must be 4-byte aligned");
  return GQA_OK;
}

// A softcap as the kernels take it: c log2(e) has to be a float, below the stand-in for minus infinity of their running
// maxima. (c tanh(s / c) is s here for every |s| below 2^87, and still grows with s beyond.)
inline float kernel_softcap(float c) { return c < 0x1p99f ? c : 0x1p99f; }

}  // namespace gqa
