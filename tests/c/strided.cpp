// Strided::overlaps against the bytes themselves, for small matrices in one buffer: two that share a byte always
// overlap; two that share none do not, where their strides are equal or one of them is a single row.
#include <cstdio>
#include <vector>

#include "strided.h"

using namespace fsdp;

int main() {
  constexpr int kBytes = 72;
  alignas(64) static unsigned char buffer[kBytes];
  std::vector<Strided> all;
  for (int size = 1; size <= 2; ++size)
    for (int rows = 1; rows <= 3; ++rows)
      for (int cols = 1; cols <= 5; cols += 2)
        for (int stride = cols; stride <= cols + 6; stride += rows == 1 ? 3 : 1)
          for (int at = 0; at + ((rows - 1) * stride + cols) * size <= kBytes && at < 40; at += size)
            all.push_back({buffer + at, rows, cols, stride, size});
  const auto bytes = [&](const Strided& m) {
    std::vector<bool> in(kBytes, false);
    for (int64_t r = 0; r < m.rows; ++r)
      for (int64_t b = 0; b < m.cols * m.size; ++b)
        in[static_cast<const unsigned char*>(m.p) - buffer + r * m.stride * m.size + b] = true;
    return in;
  };
  std::vector<std::vector<bool>> in;
  for (const Strided& m : all) in.push_back(bytes(m));
  long missed = 0, refused = 0, pairs = 0;
  for (size_t i = 0; i < all.size(); ++i)
    for (size_t k = 0; k < all.size(); ++k) {
      const Strided &a = all[i], &b = all[k];
      bool shared = false;
      for (int c = 0; c < kBytes && !shared; ++c) shared = in[i][c] && in[k][c];
      const bool said = a.overlaps(b);
      ++pairs;
      if (shared && !said) ++missed;
      if (!shared && said && (a.pitch() == b.pitch() || a.rows == 1 || b.rows == 1)) {
        if (++refused <= 5)
          std::printf("refused: %ldx%ld stride %ld size %d at %ld, %ldx%ld stride %ld size %d at %ld\n", long(a.rows), long(a.cols),
                      long(a.stride), a.size, long(static_cast<const unsigned char*>(a.p) - buffer), long(b.rows), long(b.cols),
                      long(b.stride), b.size, long(static_cast<const unsigned char*>(b.p) - buffer));
      }
    }
  std::printf("%ld pairs, %ld missed, %ld refused without need\n", pairs, missed, refused);
  return missed != 0 || refused != 0;
}
