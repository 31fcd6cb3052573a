// What the entry points of the row operators share: the checks of a matrix, and the
// row type as a template argument.
#pragma once

#include <cstdint>

#include "internal.h"
#include "rows.cuh"

namespace tbe {

inline tbe_status launched() {
  note_launch();
  return cudaGetLastError() == cudaSuccess ? TBE_OK : TBE_ECUDA;
}

// A matrix of an entry point, its row stride in elements of `bytes`.
struct Matrix {
  const void* p;
  int64_t stride;
  int bytes;
  bool good(int64_t rows, int64_t width) const {
    return p && stride >= width && aligned_to(p, bytes) &&
           (rows < 2 || stride <= INT64_MAX / 64 / rows);
  }
  Bytes span(int64_t rows, int64_t width) const {
    return {p, rows, width * bytes, rows < 2 ? width * bytes : stride * bytes};
  }
  // Whether its rows can be moved in `unit` bytes (a power of two) from end to end.
  bool vectors(int64_t width, int unit) const {
    return aligned_to(p, unit) && stride * bytes % unit == 0 && width * bytes % unit == 0;
  }
};

// Calls f with a value of the row type.
template <typename F>
tbe_status for_dtype(int32_t dtype, F f) {
  if (dtype == TBE_DT_F32) return f(float{});
  if (dtype == TBE_DT_F16) return f(__half{});
  return f(__nv_bfloat16{});
}

}  // namespace tbe
