// Goes through the 16-byte pieces that a thread's vector loads ask for, row by row: every piece
// holds an element of the row, every element is asked for, and a row that is not there (the
// rest of a warp past the last row) asks for nothing.
#include <cstdio>
#include <vector>

#include "row_map.h"

using namespace fsdp;

static int failures = 0;

static void fail(const char* what, int size, int n, int phase, int cols, int t, int j) {
  if (++failures <= 20)
    std::printf("%s: %d-byte elements, %d threads, phase %d, cols %d, thread %d, place %d\n", what, size, n, phase, cols, t, j);
}

// A row of `cols` elements (0: not there) over n threads of v groups each, as RowLoad::load asks for it.
template <RowMap kMap>
static void row(int size, int n, int v, int phase, int cols) {
  std::vector<int> seen(cols, 0);
  for (int t = 0; t < n; ++t)
    for (int k = 0; k < v; ++k) {
      const int j = place<kMap>(RowThreads{t, n, phase}, k, 0);
      const bool first = holds_some<kMap>(j, 4, cols), second = kMap == kVector ? first : holds_some<kMap>(j + 4, 4, cols);
      // 16-byte pieces: one of 8 two-byte elements, or two of 4 four-byte elements
      const int piece = 16 / size;
      for (int at = j; at < j + 8; at += piece) {
        const bool asked = size == 2 ? first || second : at == j ? first : second;
        if (!asked) continue;
        if ((at + phase) % piece != 0) fail("a piece off its boundary", size, n, phase, cols, t, at);
        bool some = false;
        for (int e = at; e < at + piece; ++e)
          if (e >= 0 && e < cols) some = true, ++seen[e];
        if (!some) fail("a piece outside the row", size, n, phase, cols, t, at);
      }
    }
  for (int e = 0; e < cols; ++e)
    if (seen[e] != 1) fail("an element not read once", size, n, phase, cols, -1, e);
}

int main() {
  for (int size = 2; size <= 4; size += 2)
    for (int phase = 0; phase < 16 / size; ++phase) {
      for (int n : {8, 16, 32, 64, 512})
        for (int v = 1; v <= 4; ++v) {
          row<kShifted>(size, n, v, phase, 0);
          const int most = n * v * 8 - 7;
          for (int cols = 1; cols <= most; cols += most < 300 || cols < 20 || cols > most - 20 ? 1 : 37)
            row<kShifted>(size, n, v, phase, cols);
        }
    }
  for (int size = 2; size <= 4; size += 2)
    for (int n : {8, 16, 32, 96})
      for (int v = 1; v <= 4; ++v)
        for (int cols = 0; cols <= n * v * 8; cols += 8) row<kVector>(size, n, v, 0, cols);
  std::printf("%d failures\n", failures);
  return failures != 0;
}
