// Host check of csrc/forms.h: the tiles that the estimates of the matrix products
// count are the tiles that cover the outputs, of one product and of two stacked
// ones (both weights' gradients of a gated block), over sizes and forms.
#include <cstdio>

#include "forms.h"

using namespace arx;

static long checks = 0;

// Tiles that cover a [rows, cols] output, counted one by one.
static uint32_t cover(uint64_t rows, uint64_t cols, uint32_t tile_rows, uint32_t tile_cols) {
  uint32_t n = 0;
  for (uint64_t r = 0; r < rows; r += tile_rows)
    for (uint64_t c = 0; c < cols; c += tile_cols) ++n;
  return n;
}

static bool same(const GemmCall& c, const Form& f) {
  const int products = c.p2 && !c.q2 ? 2 : 1;
  const uint32_t rows = f.wide ? 2 * kLanes : f.bn, cols = f.wide ? f.subs * f.bn : kLanes;
  const uint32_t want = products * cover(c.rows, c.cols, rows, cols);
  const uint32_t launched = tiles_of(c, f.wide, f.bn, f.subs).all();
  ++checks;
  if (f.tiles == want && launched == want) return true;
  std::printf("%d x [%llu, %llu], %s tiles of %u x %u: estimated %u, launched %u, cover %u\n", products,
              (unsigned long long)c.rows, (unsigned long long)c.cols, f.wide ? "wide" : "split", rows, cols, f.tiles,
              launched, want);
  return false;
}

int main() {
  bool ok = true;
  char memory = 0;
  const uint32_t sizes[] = {1, 7, 64, 65, 127, 128, 129, 200, 256, 257, 520, 1000, 1030, 1025, 2050, 2176, 4096, 4097, 8192};
  for (uint32_t rows : sizes)
    for (uint32_t cols : sizes)
      for (int stacked = 0; stacked < 2; ++stacked)
        for (int mn = 0; mn < 2; ++mn)
          for (int copies = 0; copies < 2; ++copies)
            for (uint32_t steps : {1u, 2u, 5u, 16u, 33u, 128u}) {
              GemmCall c{};
              c.rows = rows, c.cols = cols, c.p_mn = mn != 0;
              if (stacked) c.p2 = &memory;
              ok = same(c, choose_form(c, steps, true, copies != 0)) && ok;
              if (!ok) return 1;
            }
  // Every form's count, whichever is chosen.
  for (uint32_t rows = 1; rows < 600; rows += 13)
    for (uint32_t cols = 1; cols < 600; cols += 29)
      for (uint32_t bn = 16; bn <= 256; bn *= 2)
        for (int kind = 0; kind < 6; ++kind) {
          GemmCall c{};
          c.rows = rows, c.cols = cols;
          if (kind & 1) c.p2 = &memory;
          const bool wide = kind / 2 > 0;
          const uint32_t subs = kind / 2 == 2 ? 2 : 1;
          Form f{};
          f.wide = wide, f.bn = bn, f.subs = subs, f.tiles = tiles_of(c, wide, bn, subs).all();
          if (!same(c, f)) return 1;
        }
  std::printf("%ld\n", checks);
  return 0;
}
