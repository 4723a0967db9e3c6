// Host check of csrc/spans.h: every read of the kernels for rows off 16 bytes
// lies inside its matrix and brings the right bytes, over sizes, strides,
// alignments and tiles.  The matrices exist as address ranges only.
#include <algorithm>
#include <cstdio>
#include <random>
#include <vector>

#include "spans.h"

using namespace arx;

static long checks = 0;
#define CHECK(c, ...)                                    \
  do {                                                   \
    ++checks;                                            \
    if (!(c)) {                                          \
      std::printf("line %d: %s: ", __LINE__, #c);        \
      std::printf(__VA_ARGS__);                          \
      std::printf("\n");                                 \
      return false;                                      \
    }                                                    \
  } while (0)

constexpr uintptr_t kBase = uintptr_t(1) << 32;

// A row's units: inside the matrix, and every byte of the row in its place.
static bool rows_as_units() {
  for (uint32_t size : {2u, 4u})
    for (uint32_t lead = 0; lead < 16; lead += size)
      for (uint32_t cols : {1u, 2u, 3u, 5u, 7u, 8u, 9u, 15u, 16u, 17u, 31u, 33u, 250u, 257u})
        for (uint32_t pad : {0u, 1u, 2u, 3u, 5u, 7u, 8u, 9u})
          for (uint32_t rows : {1u, 2u, 3u, 9u}) {
            const uint64_t ld = (cols + pad) * size;
            const uintptr_t lo = kBase + lead, hi = lo + (rows - 1) * ld + cols * size;
            const uint32_t slot = (cols * size + 30 + 15) / 16 * 16;  // row_slot of norm.cuh
            for (uint32_t r = 0; r < rows; ++r) {
              const uintptr_t row = lo + r * ld;
              const uint32_t units = row_units(row, cols * size);
              std::vector<int> have(slot, 0);
              for (uint32_t u = 0; u < units; ++u) {
                const uintptr_t at = first_unit(row) + 16 * u, from = at < lo ? lo : at, to = at + unit_bytes(at, hi);
                CHECK(at % 16 == 0 && at + 16 > lo && at < hi && from < to && to <= at + 16, "row %u unit %u", r, u);
                CHECK(to <= hi, "row %u unit %u of %u", r, u, cols);
                CHECK(16 * u + 16 <= slot, "row %u unit %u", r, u);
                if (at < lo) CHECK((to - from) % 2 == 0 && from % 2 == 0, "element by element");
                for (uintptr_t b = from; b < to; ++b) have[16 * u + (b - at)] = 1;
              }
              for (uint32_t b = 0; b < cols * size; ++b) CHECK(have[(row & 15) + b], "row %u byte %u of %u", r, b, cols);
            }
          }
  return true;
}

// Units of an operand by loading threads.
template <int kWord>
static bool operand_units() {
  std::mt19937 rng(kWord);
  const auto pick = [&](uint32_t n) { return uint32_t(rng() % n); };
  for (int trial = 0; trial < 1500; ++trial) {
    const uint32_t mn = pick(2), rows = 1 + pick(400), k = 1 + pick(300);
    const uint32_t outer = mn ? k : rows, inner = mn ? rows : k;
    uint64_t ld = inner + pick(12);
    uint32_t lead = pick(8);
    if (kWord == 8) ld = (ld + 3) / 4 * 4, lead &= 4;  // every row on 8 bytes
    if (outer == 1) ld = inner;
    const uintptr_t lo = kBase + 2 * lead, hi = lo + ((outer - 1) * ld + inner) * 2;
    const uint32_t tile = mn ? 64u << pick(2) : 16u << pick(4), row0 = pick((rows + tile - 1) / tile) * tile;
    const Operand o = operand(reinterpret_cast<const uint16_t*>(lo), ld, mn, rows, k, row0);
    const uint32_t steps = (k + kStep - 1) / kStep, first = pick(steps);
    for (uint32_t id = 0; id < 1024; ++id) {
      Place c = place<kWord>(o, id, tile * 8, first);
      for (uint32_t i = first; i < steps; ++i, c.at += c.step) {
        const uint32_t row = unit_row(o, c.id, i * kStep), col = unit_col(o, c.id, i * kStep);
        if (c.fast && i != 0 && i + 1 != steps) {
          const uintptr_t a = reinterpret_cast<uintptr_t>(c.at), n = kWord == 8 ? 16 : c.shifted ? 20 : 16;
          CHECK(a % (kWord == 8 ? 8 : 4) == 0, "trial %d", trial);
          CHECK(a >= lo && a + n <= hi, "trial %d mn %u rows %u k %u ld %u lead %u id %u stage %u", trial, mn, rows, k,
                unsigned(ld), lead, id, i);
          // The unit itself, for the rows that the matrix has.
          if (mn || row < rows) CHECK(a + (c.shifted ? 2 : 0) == lo + (row * ld + col) * 2, "trial %d", trial);
          if (mn) CHECK(row < outer, "trial %d", trial);
        } else {
          const int n = std::min(8, unit_elements(o, row, col));
          if (n > 0) CHECK(row < outer && col + n <= inner, "trial %d id %u stage %u", trial, id, i);
          // What exists of it is taken.
          if (row < outer && col < inner) CHECK(n == int(std::min(8u, inner - col)), "trial %d", trial);
        }
      }
    }
  }
  return true;
}

// Words of a row, and the row that the lanes make of them.
static bool realigned_rows() {
  for (int64_t cols : {1, 2, 3, 5, 62, 63, 64, 65, 66, 127, 128, 129, 130, 1000, 1022, 1023, 1024, 1025, 1026, 1027, 1088, 2047,
                       2048, 2049, 2050, 2051, 4099})
    for (int lead = 0; lead < 2; ++lead)
      for (int64_t c0 = 0; c0 < cols; c0 += kRealignChunk) {
        const bool odd = lead, inside = realign_inside(c0, cols, odd);
        const int64_t rest = cols - c0;
        // Halves of a lane's words: the row's element, or -1.
        std::vector<int64_t> lo((kRealignWords + 1) * 32, -1), hi(lo);
        for (uint32_t i = 0; i <= kRealignWords; ++i)
          for (uint32_t lane = 0; lane < 32; ++lane) {
            if (i == kRealignWords && !(odd && lane == 0)) continue;
            const int64_t c = c0 + 2 * int64_t(lane + 32 * i) - odd;
            const int64_t in = realign_element(lane, i, odd);
            const uint32_t at = 32 * i + lane;
            CHECK(in == c - c0, "lane %u word %u", lane, i);
            if (!inside && 64 * int64_t(i) > rest) continue;
            if (inside || realign_both(in, c0, rest)) {
              CHECK(c >= 0 && c + 1 < cols, "cols %ld c0 %ld lane %u word %u", long(cols), long(c0), lane, i);
              lo[at] = c, hi[at] = c + 1;
            } else if (realign_lower(in, c0, rest)) {
              CHECK(c >= 0 && c < cols, "cols %ld c0 %ld lane %u word %u", long(cols), long(c0), lane, i);
              lo[at] = c;
            } else if (realign_upper(in, c0)) {
              CHECK(c == -1, "cols %ld", long(cols));
              hi[at] = 0;
            }
          }
        for (uint32_t i = 0; i < kRealignWords; ++i)
          for (uint32_t lane = 0; lane < 32; ++lane) {
            const uint32_t at = 32 * i + lane;
            const int64_t d = 2 * int64_t(at);
            if (d >= rest) continue;
            const int64_t a = odd ? hi[at] : lo[at], b = odd ? lo[at + 1] : hi[at];
            CHECK(a == c0 + d, "cols %ld c0 %ld element %ld", long(cols), long(c0), long(d));
            if (d + 1 < rest) CHECK(b == c0 + d + 1, "cols %ld c0 %ld element %ld", long(cols), long(c0), long(d));
          }
      }
  return true;
}

int main() {
  if (!rows_as_units() || !operand_units<2>() || !operand_units<8>() || !realigned_rows()) return 1;
  std::printf("%ld checks\n", checks);
  return 0;
}
