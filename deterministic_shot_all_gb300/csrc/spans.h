// What the kernels for rows off 16 bytes read and where: address arithmetic
// alone, used by the kernels and checked on the host over sizes, strides and
// alignments (a read outside a matrix may go unnoticed on a GPU).
#pragma once

#include <cstddef>
#include <cstdint>

#ifdef __CUDACC__
#define ARX_HD __host__ __device__ __forceinline__
#else
#define ARX_HD inline
#endif

namespace arx {

// ---- a row as the aligned 16-byte units that cover it (norm.cuh) ------------------------

// The first unit of a row of `bytes` bytes at address `row`, and how many cover it.
ARX_HD uintptr_t first_unit(uintptr_t row) { return row & ~uintptr_t(15); }
ARX_HD uint32_t row_units(uintptr_t row, uint32_t bytes) { return uint32_t((row + bytes - first_unit(row) + 15) >> 4); }

// Bytes of the unit at address `at` before the matrix's end `hi`.  (Those of a
// unit that begins before the matrix, at < lo, are [lo, at + unit_bytes).)
ARX_HD uint32_t unit_bytes(uintptr_t at, uintptr_t hi) { return at + 16 <= hi ? 16 : uint32_t(hi - at); }

// ---- units of 8 elements of a product's operand, loaded by threads (linear.cu) --------------

constexpr uint32_t kStep = 64;  // contraction elements in a stage

struct Operand {
  const uint16_t* p;
  uint64_t ld;
  uint32_t nrows, ncols;  // as stored
  uint32_t mn, row0;      // the tile's first matrix row
};

ARX_HD Operand operand(const uint16_t* p, uint64_t ld, uint32_t mn, uint32_t rows, uint32_t k, uint32_t row0) {
  return Operand{p, ld, mn ? k : rows, mn ? rows : k, mn, row0};
}

// Row and column of a unit in the matrix as stored, k0 the stage's first
// contraction element.
ARX_HD uint32_t unit_row(const Operand& o, uint32_t id, uint32_t k0) {
  return o.mn ? k0 + (id >> 3 & 63u) : o.row0 + (id >> 3);
}
ARX_HD uint32_t unit_col(const Operand& o, uint32_t id, uint32_t k0) {
  return (o.mn ? o.row0 + (id >> 9) * 64 : k0) + (id & 7u) * 8;
}

// The elements of a unit that exist.
ARX_HD int unit_elements(const Operand& o, uint32_t row, uint32_t col) {
  return row < o.nrows ? int(o.ncols) - int(col) : 0;
}

// One of a thread's places in the stages of a tile.  `at`, if `fast` and in any
// stage but the contraction's first and last, is where a whole unit is read:
// 16 bytes, in words of 8 (kWord = 8), or in words of 4 (kWord = 2), one more
// where the unit lies between them (`shifted`).
struct Place {
  const uint8_t* at;  // in the next stage to fetch
  uint64_t step;      // from stage to stage
  uint32_t id;
  bool on, fast, shifted;
};

// Threads beyond the operand's units fetch another's once more and store
// nothing: a load under a condition of its own is waited for where the
// condition ends, and the stages in flight with it (64 us became 127).
template <int kWord>
ARX_HD Place place(const Operand& o, uint32_t id, uint32_t units, uint32_t first) {
  Place c;
  c.on = id < units;
  c.id = c.on ? id : id % units;
  const uint32_t row = unit_row(o, c.id, first * kStep), col = unit_col(o, c.id, first * kStep);
  // Past the matrix's last row (MN-major: column) a unit feeds results that
  // are not stored: whole ones read another row instead, cut ones take the
  // general path.
  const uint32_t safe = o.mn ? row : (row < o.nrows ? row : 0);
  c.fast = o.mn ? col + 8 <= o.ncols : true;
  const uintptr_t a = reinterpret_cast<uintptr_t>(o.p + safe * o.ld + col);
  c.shifted = kWord == 2 && (a & 2) != 0;
  c.at = reinterpret_cast<const uint8_t*>(kWord == 2 ? a & ~uintptr_t(3) : a);
  c.step = o.mn ? kStep * o.ld * 2 : kStep * 2;
  return c;
}

// ---- words of a row on its way to an aligned one (realign.cu) ------------------------------

constexpr uint32_t kRealignWords = 16, kRealignChunk = 64 * kRealignWords;  // words to a lane; elements to a warp

// Does every word that a warp looks at in the chunk from column c0 on lie
// inside the row?  `odd`: the chunk starts between two words.
ARX_HD bool realign_inside(int64_t c0, int64_t cols, bool odd) {
  return (c0 > 0 || !odd) && cols - c0 >= int64_t(kRealignChunk) + odd;
}

// Where it does not: word 32 i of a lane's holds elements c and c + 1 of the
// chunk's `rest` elements.  It is read whole, or its lower half, or, before the
// row's first word, the upper one, or nothing of it.
ARX_HD int64_t realign_element(uint32_t lane, uint32_t i, bool odd) { return 2 * int64_t(lane + 32 * i) - odd; }
ARX_HD bool realign_both(int64_t c, int64_t c0, int64_t rest) { return c + c0 >= 0 && c + 1 < rest; }
ARX_HD bool realign_lower(int64_t c, int64_t c0, int64_t rest) { return c + c0 >= 0 && c < rest; }
ARX_HD bool realign_upper(int64_t c, int64_t c0) { return c + c0 == -1; }

}  // namespace arx
