// input_grad_plan.h -- how the input gradient's product [M][N] x [N][K] is cut into
// tiles and shared among pairs of blocks.  Host arithmetic without CUDA, so that
// the rule is tested for any number of SMs.
#pragma once
#include <stdint.h>

namespace sq {

constexpr int kGradTileRows = 256;  // of dx, by a pair of blocks
constexpr int kGradStep = 64;       // terms of the contraction in a stage

struct InputGradPlan {
  int bn;            // columns of a tile, 128 or 256
  int splits;        // pairs that share a tile's contraction, a cluster of 2 splits blocks
  int64_t tiles;
  int64_t clusters;  // of the grid
};

inline InputGradPlan input_grad_plan(int64_t M, int64_t N, int64_t K, int sms) {
  const int64_t mt = (M + kGradTileRows - 1) / kGradTileRows;
  const int64_t pairs = sms > 2 ? sms / 2 : 1;
  auto tiles = [&](int64_t bn) { return mt * ((K + bn - 1) / bn); };
  // Few tiles: two or four pairs share each one's contraction, where it is long
  // enough to pay for the sums' way through distributed shared memory (about 3
  // us) and all the clusters run at once: 148 SMs have room for 15 of eight blocks,
  // 33 of four, a cluster lying within one of the GPU's partitions, other numbers of
  // SMs in proportion.  200 rows, replayed graphs: 3840 -> 1920 18.0 us by four pairs,
  // 22.1 by two, 27.7 by one; 1536 -> 1536 13.5, 14.6, 15.4; 384 -> 768 10.5, 10.5, 9.1.
  // The sums of a tile take the place of the stages, so a cluster that shares one
  // has no other: as many clusters as tiles, whatever runs at once.
  const int64_t narrow = tiles(128), steps = (N + kGradStep - 1) / kGradStep;
  if (steps >= 24 && narrow * 148 <= 15 * static_cast<int64_t>(sms))
    return {128, 4, narrow, narrow};
  if (steps >= 24 && narrow * 148 <= 33 * static_cast<int64_t>(sms))
    return {128, 2, narrow, narrow};
  // Tile width: a block's time goes with the operand rows that it fetches, 128 +
  // bn / 2 a step, times the rounds of tiles.
  auto cost = [&](int64_t bn) { return (tiles(bn) + pairs - 1) / pairs * (128 + bn / 2); };
  const int bn = cost(256) <= cost(128) ? 256 : 128;
  const int64_t n = tiles(bn);
  return {bn, 1, n, n < pairs ? n : pairs};
}

}  // namespace sq
