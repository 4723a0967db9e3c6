// Which form of the matrix products on the tensor cores a call takes (linear.cu,
// gated.cu): tiles, and estimates of time.  Host code alone.
#pragma once

#include <cstdint>

#include "ops_launch.h"

namespace arx {
namespace {

constexpr uint32_t kLanes = 128;  // rows of P in a tile (accumulator lanes)

inline uint32_t ceil_div(uint64_t a, uint64_t b) { return uint32_t((a + b - 1) / b); }

// Which form, with how many rows of Q to a tile and how many blocks to a
// tile's contraction: the one with the least estimated time, in SM cycles, on
// 152 SMs (a constant: the form decides the order of a sum).
struct Form {
  bool wide;
  uint32_t bn, split, subs, tiles;
  double cycles;
};

// Tiles of a product in either direction.  Of two stacked products the second's
// rows begin with a tile of their own.  The estimates and the launches count by it.
struct Tiles {
  uint32_t rows, cols;
  uint32_t all() const { return rows * cols; }
};
inline Tiles tiles_of(const GemmCall& c, bool wide, uint32_t bn, uint32_t subs) {
  const uint32_t products = c.p2 && !c.q2 ? 2 : 1;
  return {products * ceil_div(c.rows, wide ? 2 * kLanes : bn), ceil_div(c.cols, wide ? subs * bn : kLanes)};
}

// (allow_wide: false leaves the wide forms out; join_more: cycles more for a row of Q
// that a split block joins and stores, shared out over its cluster.)
inline Form choose_form(const GemmCall& c, uint32_t steps, bool p_copy, bool q_copy, bool allow_wide = true,
                        double join_more = 0) {
  constexpr uint32_t sms = 152;
  Form best{};
  const auto consider = [&](const Form& f) {
    if (best.bn == 0 || f.cycles < best.cycles) best = f;
  };
  // A stage of `rows` rows of c.p and `cols` of c.q costs its copies or its
  // products (2.1 cycles a row of the kernel's Q), whichever is longer.
  // Measured, bytes a cycle into an SM: 46 in pairs when all of them are at
  // work, 53 for half of them, a seventh less with 128 rows of Q; 41 for a
  // split block alone on its SM, 55 for one with the whole shared memory, 66 for
  // two; through loading threads 16 (12 in pairs, where the slower of two blocks
  // counts).
  const bool threads = !p_copy || !q_copy;
  const auto stage = [&](uint32_t rows, uint32_t cols, uint32_t bn, double engine, double loaded) {
    const double copies = rows * 128.0 / (p_copy ? engine : loaded) + cols * 128.0 / (q_copy ? engine : loaded);
    return copies > 2.1 * bn ? copies : 2.1 * bn;
  };
  const bool stacked = c.p2 && !c.q2;
  // Starting and ending a block takes about 6000 cycles, joining and storing a
  // tile 25 a row of Q, 30 to 40 through a cluster; of a wide tile all but the last
  // run under the next one's products, 2800 + 7 a row at the least.
  // Of stacked products, whose contraction is the tokens and whose outputs are the
  // weights, most of a split block's time is the storing: 60 a row more.  Over 88
  // sizes, 1 to 7,909 tokens, the forms chosen take 1.04 of the best ones' time in
  // the mean and 1.28 at most, without it 1.15 and 2.27.  Both gradients of
  // [2048, 1024] from 64 tokens: wide 8.2 us, split 14.1 and more; of [96, 2832] from
  // 1178: split 10.9, wide 13.9.
  constexpr uint32_t pairs = sms / 2;
  for (uint32_t bn = 256; bn >= 128 && allow_wide; bn /= 2) {
    const uint32_t tiles = tiles_of(c, true, bn, 1).all();
    const double engine = (58 - 12.0 * (tiles < pairs ? tiles : pairs) / pairs) * (bn == 128 ? 0.86 : 1);
    const double products = steps * stage(kLanes, bn / 2, bn, engine, 12), store = 2800 + 7 * bn;
    consider({true, bn, 1, 1, tiles, ceil_div(tiles, pairs) * (products > store ? products : store) + 6000 + 25 * bn});
  }
  // Two accumulators to a tile: 1290 cycles a stage (630 us against 681 at
  // 8192^3, where the card's power sets the clock), and no tile's epilogue runs
  // under the next one's products.
  if (!threads && allow_wide) {
    const uint32_t tiles = tiles_of(c, true, 256, 2).all(), rest = tiles % pairs;
    const bool halves = rest && 2 * rest <= pairs;
    const double rounds = tiles / pairs + (rest && !halves);
    consider({true, 256, 1, 2, tiles,
              rounds * (steps * 1290.0 + 4000) + (halves ? steps * 712.0 + 4000 : 0) + 6000 + 25 * 256});
  }
  for (uint32_t bn = c.p_mn ? 64 : 16; bn <= (threads ? 128 : 256); bn *= 2) {
    const uint32_t tiles = tiles_of(c, false, bn, 1).all();
    const bool two = !threads && bn <= 128;  // blocks to an SM
    for (uint32_t split = 1; split <= 8 && (split == 1 || split <= steps); split *= 2) {
      // Clusters at work at once: those of 4 and 8 leave some SMs of a processing
      // cluster over.
      const uint32_t at_once = two ? (split == 8 ? 36 : split == 4 ? 72 : 2 * sms / split)
                                   : (split == 8 ? 14 : split == 4 ? 36 : sms / split);
      const double join = ((split == 8 ? 40 : split > 1 ? 30 : 25) +
                           (two && !stacked ? 0 : (stacked ? 60 : join_more) / split)) * bn;
      const uint32_t rounds = ceil_div(tiles, at_once);
      const double on_sm = !two ? rounds : rounds > 1 ? 2 * rounds : ceil_div(uint64_t(tiles) * split, sms);
      const double engine = two && on_sm > 1 ? 66 : bn > 128 ? 55 : 41;
      const double own = ceil_div(steps, split) * stage(bn, kLanes, bn, engine, 16) + join;
      consider({false, bn, split, 1, tiles, two ? on_sm * own + 6000 : on_sm * (own + 6000)});
    }
    if (bn >= c.rows) break;
  }
  return best;
}

}  // namespace
}  // namespace arx
