// api_util.cuh -- argument-checking helpers shared by the C ABI translation units.
#pragma once

#include "../../include/qnre.h"

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

namespace qnre {
namespace api {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct ByteRange {
  uintptr_t lo, hi;  // [lo, hi); empty when lo == hi
};

inline bool overlaps(ByteRange a, ByteRange b) { return a.lo < b.hi && b.lo < a.hi; }

inline ByteRange span(const void* p, uint64_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {lo, lo + static_cast<uintptr_t>(bytes)};
}

inline int dtype_size(int32_t dt) {
  switch (dt) {
    case QNRE_DTYPE_BF16: return 2;
    case QNRE_DTYPE_FP16: return 2;
    case QNRE_DTYPE_FP32: return 4;
    default: return 0;
  }
}

inline qnre_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? QNRE_OK : QNRE_ERR_CUDA; }

// Checks common to every strided rank-4 view; fills the byte span of its
// storage.  Extents 0 and 1 (batch, sequence) may be 0 (an empty call).
inline qnre_status_t check_view(const qnre_tensor4_t* t, ByteRange* range) {
  if (t == nullptr || t->data == nullptr) return QNRE_ERR_INVALID_ARG;
  const int esz = dtype_size(t->dtype);
  if (esz == 0) return QNRE_ERR_UNSUPPORTED;
  bool empty = false;
  uint64_t last = 0;
  for (int i = 0; i < 4; ++i) {
    if (t->shape[i] < (i < 2 ? 0 : 1) || t->stride[i] < 1) return QNRE_ERR_INVALID_ARG;
    if (t->shape[i] > (int64_t{1} << 40) || t->stride[i] > (int64_t{1} << 40)) return QNRE_ERR_CAPACITY;
    if (t->shape[i] == 0) {
      empty = true;
      continue;
    }
    last += static_cast<uint64_t>(t->shape[i] - 1) * static_cast<uint64_t>(t->stride[i]);
    if (last > (uint64_t{1} << 56)) return QNRE_ERR_CAPACITY;
  }
  if (!aligned(t->data, static_cast<uintptr_t>(esz))) return QNRE_ERR_ALIGNMENT;
  *range = empty ? ByteRange{0, 0} : span(t->data, (last + 1) * static_cast<uint64_t>(esz));
  return QNRE_OK;
}

// Head rows of this view can be copied as 16-byte vectors.
inline bool rows_vectorisable(const qnre_tensor4_t* t, int esz) {
  if (t->stride[3] != 1) return false;
  if ((t->shape[3] * esz) % 16 != 0) return false;
  if (!aligned(t->data, 16)) return false;
  for (int i = 0; i < 3; ++i)
    if ((t->stride[i] * esz) % 16 != 0) return false;
  return true;
}

// Whether two views of one element size share an element.  q and k are often bands of one buffer, token-major or head-major,
// so their spans meet although no element does.  A common element means that the distance of the bases is a sum of whole
// steps, of each axis from -(b's extent - 1) to a's (where both step alike, else each its own).  From the longest
// step down only those counts are tried that the shorter steps can make up for: one or two an axis where strides nest.
// After kOverlapTries counts (strides that do not nest) the views are taken to meet.
constexpr int kOverlapTries = 4096;

struct Step {
  int64_t stride, lo, hi, rest;  // rest: how far the shorter steps reach
};

inline bool steps_reach(const Step* s, int n, int64_t d, int* tries) {
  if (n == 0) return d == 0;
  auto floor_div = [](int64_t a, int64_t b) { return a >= 0 ? a / b : -((-a + b - 1) / b); };
  const int64_t lo = std::max(s->lo, -floor_div(s->rest - d, s->stride));
  const int64_t hi = std::min(s->hi, floor_div(s->rest + d, s->stride));
  for (int64_t i = lo; i <= hi; ++i) {
    if (--*tries < 0 || steps_reach(s + 1, n - 1, d - i * s->stride, tries)) return true;
  }
  return false;
}

inline bool views_overlap(const qnre_tensor4_t* a, ByteRange ra, const qnre_tensor4_t* b, ByteRange rb) {
  if (!overlaps(ra, rb)) return false;
  const int esz = dtype_size(a->dtype);
  const int64_t bytes = static_cast<const char*>(b->data) - static_cast<const char*>(a->data);
  if (esz != dtype_size(b->dtype) || bytes % esz != 0) return true;
  Step s[8];
  int n = 0;
  for (int i = 0; i < 4; ++i) {
    const int64_t na = a->shape[i] - 1, nb = b->shape[i] - 1;
    if (na > 0 && nb > 0 && a->stride[i] == b->stride[i]) {
      s[n++] = {a->stride[i], -nb, na, 0};
    } else {
      if (na > 0) s[n++] = {a->stride[i], 0, na, 0};
      if (nb > 0) s[n++] = {b->stride[i], -nb, 0, 0};
    }
  }
  std::sort(s, s + n, [](const Step& x, const Step& y) { return x.stride > y.stride; });
  for (int i = n - 2; i >= 0; --i) s[i].rest = s[i + 1].rest + std::max(-s[i + 1].lo, s[i + 1].hi) * s[i + 1].stride;
  int tries = kOverlapTries;
  return steps_reach(s, n, bytes / esz, &tries);
}

}  // namespace api
}  // namespace qnre
