// Which scale bytes the products of block-128 FP8 operands may touch: every
// access of the wide tiles' and the decode kernel's scale loads, for operands
// that are views at every offset of wider matrices, against the bound that the
// kernels give their buffer resources.  Exits 0 when no access that the bound
// lets through leaves the view's last line, and none that is needed is cut.
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "fp8_internal.h"

static long failures = 0, touched = 0;

// One lane's load of `unit` bytes at `offset` of a resource that starts at the
// scale of row `first`: the hardware drops it if its end passes the extent.
static void load(int64_t kb, int64_t ld, int64_t rows, int64_t first, int64_t line, int64_t row, int unit) {
  const int64_t offset = line * ld + row - first;
  const bool through = offset + unit <= mxfp4::fp8_scale_extent(kb, ld, rows, first, unit);
  // the view's memory ends with the last line's last row, in whole words of 4 bytes for loads of words
  const int64_t end = (kb - 1) * ld + (unit == 4 ? (rows + 3) / 4 * 4 : rows);
  if (through && first + offset + unit > end) failures++;
  if (!through && row < rows) failures++;
  touched += through;
}

int main() {
  for (int64_t rows : {1, 2, 3, 5, 16, 31, 100, 127, 128, 129, 255, 256, 257, 300, 384, 5504})
    for (int64_t pitch : {0, 16, 128, 2048})
      for (int64_t kb : {1, 2, 3, 7}) {
        const int64_t ld = (rows + 15) / 16 * 16 + pitch;
        // wide tiles: 256 rows from every multiple of 128 (a half tile), 4 bytes a lane
        for (int64_t first = 0; first < rows; first += 128)
          for (int64_t line = 0; line < kb; line++)
            for (int lane = 0; lane < 64; lane++) load(kb, ld, rows, first, line, first + 4 * lane, 4);
        // decode: 16 rows of the weights, 16 to 128 of the activations, a byte a lane
        for (int tile : {16, 32, 64, 128})
          for (int64_t first = 0; first < rows; first += tile)
            for (int64_t line = 0; line < kb; line++)
              for (int r = 0; r < tile; r++) load(kb, ld, rows, first, line, first + r, 1);
      }
  // gated: 128 rows of either weight of a pair [2 np, k], lanes 32 and up in the second
  for (int64_t np : {128, 256, 5504})
    for (int64_t kb : {1, 3})
      for (int64_t first = 0; first < np; first += 128)
        for (int64_t line = 0; line < kb; line++)
          for (int lane = 0; lane < 64; lane++)
            load(kb, 2 * np, 2 * np, first, line, first + 4 * lane + (lane >= 32 ? np - 128 : 0), 4);
  // nothing to read: no rows from `first` on, or no contraction
  if (mxfp4::fp8_scale_extent(3, 64, 64, 64, 4) != 0 || mxfp4::fp8_scale_extent(0, 64, 64, 0, 1) != 0) failures++;
  if (failures) std::fprintf(stderr, "%ld accesses out of place\n", failures);
  else std::printf("%ld accesses in place\n", touched);
  return failures != 0;
}
