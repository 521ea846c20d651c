// Which kernel a product takes, by its sizes: an estimate of each kernel's time
// (in ns, from measurements on MI355X of 30 to 40 sizes a call; what decides is
// their ratio near the borders) and the least of them.
//
//   FEW    workgroups of 64 rows x 16 or 32 columns that deal the summed index among their
//          wavefronts: little latency, every operand read straight from memory
//   SMALL  tiles of 64 x 128
//   GROUP  (gated block) tiles of 128 x one group of 128 columns: the codes
//          made in the tile, no second launch
//   LARGE  tiles of 256 x 256
//
// 4096 x 8192 x 3584 (bf16 results): FEW 613 us, SMALL 195, LARGE 119; 512 x 2048 x
// 4096: 26, 22, 59; 129 x 264 x 7040: 18, 37, 94.  The gated forward, 8192 -> 3584: 64 tokens
// 37, 64, GROUP 130, 193; 512 tokens 166, 87, 135, 194; 1024 tokens 319, 171, 132, 200; 4096
// tokens LARGE 404.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace tpmlp {

enum G8Form { G8_FEW, G8_SMALL, G8_GROUP, G8_LARGE };

inline int64_t g8_over(int64_t n, int64_t d) { return (n + d - 1) / d; }

// A launch has fewer than 2^32 threads in a dimension: workgroups (of 512 at most) go in
// launches of 2^22, `launch(first, count)` each, until one fails
constexpr int64_t G8_LAUNCH = (int64_t)1 << 22;
template <typename F>
auto g8_in_launches(int64_t blocks, F launch) {
  decltype(launch(blocks, blocks)) r{};
  for (int64_t first = 0; first < blocks && r == decltype(r){}; first += G8_LAUNCH)
    r = launch(first, std::min(G8_LAUNCH, blocks - first));
  return r;
}

// FEW: 32 columns a workgroup halve the reads of A, where there are enough
// workgroups to hide their longer turns (512 x 1024 x 1024: 7.5 against 6.3 us;
// 1024 x 256 x 4096, 256 workgroups of 16 columns: 12 against 16)
inline bool g8_wide(int64_t M, int64_t N) { return M > 32 && g8_over(M, 64) * g8_over(N, 16) > 320; }

// kt: groups of the summed index, every part's; ends: what a workgroup's start and end take, in
// groups (2100 x 2056 x 384: FEW 17.6 us, SMALL 10.6); in the gated block that is the fp32 values' way through
// memory and their codes (8192 tokens, 128 -> 3584: forward FEW 175, LARGE 87; backward 194, 128)
inline double g8_few_ns(int64_t M, int64_t N, int64_t kt, int64_t ends, double wide_unit, double unit, double turn, double wide_turn) {
  const bool wide = g8_wide(M, N);
  const double units = (double)g8_over(M, 64) * g8_over(N, 16) * (kt + ends), turns = (double)g8_over(kt, 8);
  return std::max(units * (wide ? wide_unit : unit), turns * (wide ? wide_turn : turn));
}

// SMALL: two workgroups share a compute unit
inline double g8_small_ns(int64_t tiles, int64_t kt, double first, double one, double turn, double two) {
  return tiles <= 256 ? first + kt * one : 6000 + g8_over(tiles, 512) * (turn + kt * two);
}

// f32: fp32 results (their products are of bf16 on the matrix cores); large:
// whether there is a LARGE kernel
inline G8Form g8_plan_gemm(int64_t M, int64_t N, int64_t kt, bool f32, bool large) {
  if (M <= 64) return G8_FEW;
  const double few = 4000 + g8_few_ns(M, N, kt, 2, 0.64, 1.06, 2000, 1800);
  const double small = f32 ? g8_small_ns(g8_over(M, 64) * g8_over(N, 128), kt, 4000, 850, 1200, 1350)
                           : g8_small_ns(g8_over(M, 64) * g8_over(N, 128), kt, 2500, 700, 1000, 880);
  // (a tile's first loads and its store count: 4096 x 2048 x 512 19 us by LARGE, 14 by SMALL; 8192 x 8192 x 256 62 and 71)
  const double whole = 3000 + (f32 ? 13000 + kt * 2900.0 : 8000 + kt * 1700.0) * g8_over(g8_over(M, 256) * g8_over(N, 256), 256);
  if (large && whole < std::min(few, small)) return G8_LARGE;
  return few < small ? G8_FEW : G8_SMALL;
}

inline G8Form g8_plan_glu(int64_t N, int64_t F, int64_t kt, bool backward) {
  if (N <= 64) return G8_FEW;
  const int64_t fb = backward ? 128 : 64;  // columns of F a SMALL tile has
  const double few = backward ? 9000 + g8_few_ns(N, F, kt, 4, 0.95, 1.12, 2000, 2900) : 10500 + g8_few_ns(N, F, kt, 4, 1.45, 1.45, 2300, 2300);
  const double small = backward ? g8_small_ns(g8_over(N, 64) * g8_over(F, fb), kt, 15000, 870, 16000, 1350)
                                : g8_small_ns(g8_over(N, 64) * g8_over(F, fb), kt, 13000, 800, 6000, 1200);
  const double group = (backward ? 13500 + kt * 1400.0 : 11000 + kt * 1930.0) * g8_over(g8_over(N, 128) * g8_over(F, 128), 256);
  const double whole = ((backward ? 45000 : 16000) + kt * 3200.0) * g8_over(g8_over(N, 256) * g8_over(F, 2 * fb), 256);
  const double least = std::min(std::min(few, small), std::min(group, whole));
  return least == whole ? G8_LARGE : least == group ? G8_GROUP : least == small ? G8_SMALL : G8_FEW;
}

}  // namespace tpmlp
