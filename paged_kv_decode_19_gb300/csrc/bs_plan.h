// Host-only: the grid of a block-scaled decode that is planned on the device.
#pragma once

namespace pd {

// A segment (sequence, KV head, slice of 8 query columns) within a block is merged in shared
// memory; one that crosses blocks costs about as much as kCrossTiles tiles of a warp more (a fence,
// an atomic and two trips to L2: 64 rows alone took 6.8 us in one block and 11.9 us across four).
constexpr int kCrossTiles = 10;

// Blocks of the balanced schedule when the sequences' lengths are known on the device alone:
// `grid`, a full wave, or as many equal shares as there are segments, by the mean length (even
// sequences then fall on block borders, and uneven ones are still shared equally).
//   n_z slices of a KV head's columns, zg of them side by side in a block (one line of the schedule);
//   tiles: of 16 rows, of all sequences and one KV head; `wave` resident blocks of `warps`.
// With m lines a block, m the smallest divisor of the lines of a (sequence, KV head) that `grid`
// allows, a warp takes m zg / warps of a segment's tiles.  That may be above a warp's equal share of
// everything by what the crossings cost: those of a line's zg segments, or for m > 1 of two.
// Measured (8 KV heads, even sequences; full wave / this rule, us): 5 slices of 640 rows, B 1 17.0 / 13.6,
// B 4 22.6 / 15.7; 3 slices of 640 rows, B 8 23.7 / 15.9, B 16 (m = 3) 28.8 / 26.9; 2 slices of 640 rows,
// B 1 32.6 / 19.5; a block for all five slices of 640 rows, B 8, would take 35.9 where the wave takes 27.3.
inline int bs_device_grid(long long B, int H_kv, int n_z, int zg, long long tiles, int wave, int warps, int grid) {
  const int lines = n_z / zg;  // of a (sequence, KV head)
  if (B * H_kv >= grid) return grid;
  int m = 1;
  while (lines % m != 0 || B * H_kv * (lines / m) > grid) ++m;  // (m = lines fits)
  const long long budget = (long long)kCrossTiles * (m > 1 ? 2 : zg);
  if (tiles * m * zg / B / warps > tiles * H_kv * n_z / ((long long)wave * warps) + budget) return grid;
  return (int)(B * H_kv * (lines / m));
}

}  // namespace pd
