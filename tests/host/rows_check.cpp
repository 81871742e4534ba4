// Host check of the rows a tensor map takes from an allocation (pa_schedule.h): all
// that fit whole behind the pool's address, none outside.
#include <stdio.h>

#include <initializer_list>

#include "pa_schedule.h"

int main() {
  using pa::rows_behind;
  const uint64_t start = 0xfff88cc00000ull, size = 2u << 20;
  for (uint64_t off : {uint64_t(0), uint64_t(16), uint64_t(512), size - 4096, size - 16, size - 1})
    for (uint64_t row : {uint64_t(128), uint64_t(256), uint64_t(768), uint64_t(2048), uint64_t(2560)}) {
      const uint64_t rows = rows_behind(start, size, start + off, row);
      if (off + rows * row > size || off + (rows + 1) * row <= size) return 1;
    }
  if (rows_behind(start, size, start - 1, 256) || rows_behind(start, size, start + size, 256) ||
      rows_behind(0, 0, 16, 256))
    return 2;
  if (rows_behind(start, uint64_t(1) << 40, start + 256, 128) != uint64_t(1) << 31) return 3;
  printf("ok\n");
  return 0;
}
