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

// Grid of the tile kernel: `total` tiles, x * y workgroups (a grid dimension has
// fewer than 2^32 threads).
struct MxTileGrid {
  int64_t total;
  unsigned x, y;
};
constexpr MxTileGrid mx_tile_grid(int m, int n, int side) {
  const int64_t total = (int64_t)mx_groups(m, side) * mx_groups(n, side);
  const int64_t x = total < (1 << 20) ? total : 1 << 20;
  return {total, (unsigned)x, (unsigned)((total + x - 1) / x)};
}

}  // namespace k3moe
