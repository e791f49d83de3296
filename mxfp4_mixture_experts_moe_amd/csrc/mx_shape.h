// Launch arithmetic of the microscaled products: plain C++ without HIP, used by
// the launches and by the kernels themselves.
#pragma once

#include <stdint.h>

namespace k3moe {

// Groups or tiles of `side` that n >= 1 rows or columns take.  n goes up to
// 2^31 - 1, where the sum n + side - 1 would no longer fit 32 bits.
constexpr int mx_groups(int n, int side) { return (n - 1) / side + 1; }

// Grid of the few-row kernel over the groups of 16 weight rows, `side` groups
// side by side in a workgroup: the fewest rounds that two workgroups per CU
// allow, and as few workgroups as that leaves (all have the same number of
// rounds, and A is staged less often).
struct MxFewGrid {
  int rounds;
  int64_t wgs;
};
constexpr MxFewGrid mx_few_grid(int n, int side, int cus) {
  const int groups = mx_groups(n, 16), most = 2 * cus * side;
  const int rounds = (groups + most - 1) / most;
  const int64_t each = (int64_t)rounds * side;
  return {rounds, (groups + each - 1) / each};
}
// Rounds of such a workgroup, as the kernel counts them.
constexpr int mx_few_rounds(int n, int side, int wgs) {
  const int step = wgs * side;
  return (mx_groups(n, 16) + step - 1) / step;
}

// Whether the few-row kernel takes up to 16 rows of 8 bits in `chunks`, each of
// which reads all weights, and has a CU to itself for 16 of their rows; else tiles of
// 32 x 64 take them, in one pass.  A tile takes as long as three rounds of such
// workgroups (four of them hold a tile's weight rows), as six where K is no multiple
// of 512 (not `whole`).  us in chunks and in tiles: 16 x 4096 x 12288 (two chunks, 64
// tiles) 18 and 19, 16 x 7168 x 9216 (two, 112) 23 and 15, 12 x 4096 x 33792
// (three, 64) 51 and 56, 16 x 7168 x 33792 (four, 112) 103 and 58, 16 x 16384 x 65536
// (eight, 256) 947 and 132; 16 x 9000 x 16416 (two, 141) 50 and 52, 16 x 7168 x 33760
// (four, 112) 120 and 99.
constexpr bool mx8_few_in_chunks(int n, int64_t chunks, bool whole, int cus) {
  return chunks == 1 || chunks * mx_groups(n, 64) <= (whole ? cus - cus / 4 : cus + cus / 2);
}

// Grid of the tile kernel: `total` tiles, x * y workgroups (a grid dimension has
// fewer than 2^32 threads).
struct MxTileGrid {
  int64_t total;
  unsigned x, y;
};
constexpr MxTileGrid mx_tile_grid(int m, int n, int rows, int columns) {
  const int64_t total = (int64_t)mx_groups(m, rows) * mx_groups(n, columns);
  const int64_t x = total < (1 << 20) ? total : 1 << 20;
  return {total, (unsigned)x, (unsigned)((total + x - 1) / x)};
}
constexpr MxTileGrid mx_tile_grid(int m, int n, int side) { return mx_tile_grid(m, n, side, side); }

}  // namespace k3moe
