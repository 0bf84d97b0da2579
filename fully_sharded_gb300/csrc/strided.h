// Row-strided matrices in caller memory: validation and overlap checks of the
// training operators' entry points (host only).
#pragma once

#include <algorithm>
#include <cstdint>
#include <vector>

#include "fsdp.h"

namespace fsdp {

inline int size_of_dtype(int32_t dtype) {
  switch (dtype) {
    case FSDP_DTYPE_F32: case FSDP_DTYPE_I32: return 4;
    case FSDP_DTYPE_BF16: return 2;
    case FSDP_DTYPE_E4M3: return 1;
    case FSDP_DTYPE_I64: return 8;
    default: return 0;
  }
}

// A row-major matrix at `p`: rows of `cols` elements of `size` bytes, `stride` elements apart.
struct Strided {
  const void* p;
  int64_t rows, cols, stride;
  int size;

  bool ok() const {
    if (!p || reinterpret_cast<uintptr_t>(p) % size != 0) return false;
    // the span fits the address arithmetic; a single row's stride is not used
    return rows < 2 || (stride >= cols && stride <= INT64_MAX / 8 / rows);
  }
  int64_t pitch() const { return rows > 1 ? stride * size : 0; }
  uintptr_t lo() const { return reinterpret_cast<uintptr_t>(p); }
  uintptr_t hi() const { return lo() + static_cast<uintptr_t>((rows > 1 ? (rows - 1) * pitch() : 0) + cols * size); }
  bool same_place(const Strided& o) const {
    return p == o.p && size == o.size && rows == o.rows && cols == o.cols && pitch() == o.pitch();
  }
  // True when some byte belongs to both. Column slices of one buffer (equal
  // pitch, or a single row beside a matrix; columns apart) do not overlap although their spans do.
  bool overlaps(const Strided& o) const {
    if (rows < 1 || o.rows < 1 || hi() <= o.lo() || o.hi() <= lo()) return false;
    const int64_t s = std::max(pitch(), o.pitch());
    if (s == 0 || (pitch() && o.pitch() && pitch() != o.pitch())) return true;
    const int64_t d = static_cast<int64_t>((o.lo() - lo()) % static_cast<uintptr_t>(s));
    const int64_t at = o.lo() >= lo() ? d : (s - static_cast<int64_t>((lo() - o.lo()) % static_cast<uintptr_t>(s))) % s;
    return !(at >= cols * size && at + o.cols * o.size <= s);
  }
};

}  // namespace fsdp
