// Which kernel, tile and K split an e4m3 product takes (host arithmetic on its sizes alone).
#pragma once
#include "dense_plan.h"

namespace q4 {

// y = x W^T; dx = dy W; dW = dy^T x.
enum Fp8Mode { FP8_Y = 0, FP8_DX = 1, FP8_DW = 2 };

// A launch holds fewer workgroups than this (of up to 512 threads: below 2^32 in all).
constexpr int64_t kMostItems = int64_t(1) << 23;

// K slices of each tile of a last round (by expert) that leaves `room` workgroups per tile: at least
// 4 steps each, 8 at most.
constexpr int fp8_tail_slices(int64_t room, int steps) {
  const int most = steps / 4 < 8 ? steps / 4 : 8;
  return room < most ? int(room) : most;
}
// (From K = 4096 on: 32 experts of 128 rows and one of 300, 7168 / 4096, 298 -> 257 us; but 8 of 1024
// rows, 2048 / 4096, 102 -> 106, and 16 of 312, 1024 / 2048, 27 -> 31: the slices' join is a launch.)
inline bool fp8_has_tail(const Plan& p, Fp8Mode mode, int64_t steps, bool grouped) {
  return grouped && mode != FP8_DW && p.tile >= 128 && steps >= 32;
}

// Estimated time (us) of `batches` products with square tiles of `bm` and K in `ks` slices of whole
// 128-element steps: the form of plan_us, its constants (per mode and tile: a step of a workgroup
// alone on its CU and of a full CU per workgroup, a workgroup's start and end) fitted to 210
// products (17 to 4096 rows, widths 512 to 16384), whose tiles and slices were all timed: the
// plan's choice is the fastest or within 8 % of it for 204 of them (the worst 17 %, dx of 64 rows,
// 2048 / 512).  Weights from memory take at least their bytes at 5.8 TB/s.  (By expert a split last
// round is not in the estimate: how many tiles it has the offsets say.)
inline double fp8_plan_us(Fp8Mode mode, int64_t m, int64_t n, int64_t steps, int64_t batches, int bm, int64_t ks,
                          bool uneven = false) {
  const int t = bm == 64 ? 0 : bm == 128 ? 1 : 2;
  static const int held[3] = {3, 2, 1};   // workgroups a CU holds
  static const double alone[3][3] = {{0.39, 0.77, 1.30}, {0.42, 0.78, 0.81}, {0.40, 0.79, 0.84}};
  static const double full[3][3] = {{0.25, 0.51, 1.05}, {0.31, 0.53, 1.41}, {0.27, 0.62, 1.85}};
  static const double ends[3][3] = {{2.5, 3.9, 6.2}, {3.3, 4.1, 6.9}, {3.7, 6.0, 10.9}};
  static const double join[3][3] = {{3.0, 0.45, 3.6e6}, {2.5, 0.39, 3.4e6}, {2.0, 0.18, 3.5e6}};
  const int64_t per = ceil_div(steps, ks);
  // (`uneven`: m rows on average, whose tiles end with half a tile)
  const int64_t row_tiles = uneven && m > bm ? (batches * (2 * m + bm) + 2 * bm - 1) / (2 * bm) : ceil_div(m, bm) * batches;
  const int64_t wgs = row_tiles * ceil_div(n, bm) * ceil_div(steps, per);
  if (wgs >= kMostItems || (ks > 1 && m * ceil_div(n, 4) >= int64_t(1) << 32)) return 1e300;
  const int64_t rounds = ceil_div(wgs, 256 * held[t]);
  const int64_t last = std::min<int64_t>(held[t], ceil_div(wgs - (rounds - 1) * 256 * held[t], 256));
  const auto slice = [&](int64_t on_cu) {
    return ends[mode][t] + per * std::max(alone[mode][t], full[mode][t] * on_cu);
  };
  double us = (rounds - 1) * slice(held[t]) + slice(last);
  if (ks > 1) us += join[mode][0] + join[mode][1] * ks + double(ks) * m * n * 4 / join[mode][2];
  return mode == FP8_DW ? us : std::max(us, double(batches) * n * steps * 128 / 5.8e6);
}

// The few-rows kernel of y, m rows by each of `batches` matrices (fitted to 25 products of 17 to 128
// rows): a wave's chain of K steps, or the weights and the rows that each 16 columns read again.
inline double fp8_rows_us(int64_t m, int64_t k, int64_t n, int64_t batches) {
  return 3.2 + std::max(ceil_div(k, 1024) * (0.6 + 0.025 * m), double(batches) * n * k / 1e6 * (0.15 + 0.0068 * m));
}

// By expert only the device knows which experts have rows.  The few-rows kernel gets a workgroup per
// expert and 16 columns, or per run of rows that may not be empty, `runs` of them at most, and each
// workgroup searches for its run: a workgroup of an expert without a row costs 0.7 ns, a search 0.9 us
// per 512 experts in every round of 1024 workgroups (8 rows of 256 experts, 7168 / 4096: 67 us for all
// experts, 42 with the search; 300 rows of 300, 256 / 4096: 125 and 191).
inline double fp8_idle_us(int64_t runs, int64_t e, int64_t n) { return double(e - runs) * ceil_div(n, 16) * 0.7e-3; }
inline double fp8_search_us(int64_t runs, int64_t e, int64_t n) {
  return std::max(1.0, double(runs) * ceil_div(n, 16) / 1024) * 0.9 * ceil_div(e, 512);
}
inline bool fp8_rows_search(int64_t t, int64_t n, int64_t e) {
  const int64_t runs = std::min(e, t);
  return e * ceil_div(n, 16) >= kMostItems || fp8_idle_us(runs, e, n) > fp8_search_us(runs, e, n);
}
// Workgroups of the few-rows kernel (e = 1 without offsets).
inline int64_t fp8_rows_grid(int64_t t, int64_t n, int64_t e) {
  return (fp8_rows_search(t, n, e) ? std::min(e, t) : e) * ceil_div(n, 16);
}

// Calls of up to this many rows take the few-rows kernel, which multiplies without the narrow
// instructions' loss, whatever is faster: 0.5 to 1.26 times the tiles' time (one row,
// 256 / 4096, 4.6 -> 3.7 us; 16 rows, 256 / 512, 4.6 -> 2.9, 8192 / 8192 20.2 -> 21.2, 16384 / 1000 14.5
// -> 17.2, 7168 / 16384 28.4 -> 34.4; 8 rows of 8 experts, 256 / 512, 5.7 -> 3.0, of 1024, 256 / 4096,
// 9.9 -> 12.3).
constexpr int64_t kWideRows = 16;

// Whether the few-rows kernel takes 16 rows a pass, else 64.
inline bool fp8_rows_sixteen(int64_t t, int32_t e, bool grouped) {
  return t <= kWideRows || (grouped && t <= 4 * int64_t(e));
}

inline Plan fp8_tiles(Fp8Mode mode, int64_t m, int64_t n, int64_t steps, int64_t batches, bool split, double* us,
                      bool uneven = false) {
  Plan best{64, 1};
  *us = 1e301;
  for (const int bm : {64, 128, 256})
    for (const int ks : {1, 2, 3, 4, 6, 8, 12, 16}) {
      if (ks > 1 && (!split || steps / ks < 2)) break;
      const double u = fp8_plan_us(mode, m, n, steps, batches, bm, ks, uneven);
      if (u < *us) *us = u, best = Plan{bm, int(ceil_div(steps, ceil_div(steps, ks)))};
    }
  return best;
}

// The product over t rows in all, e matrices of them with `grouped`; by expert the rows are known
// by their number alone (the offsets are on the device).
inline Plan fp8_plan(Fp8Mode mode, int64_t t, int64_t k, int64_t n, int32_t e, bool grouped) {
  if (mode == FP8_Y && t <= kWideRows) return Plan{0, 1};
  double us;
  const int64_t rows = grouped ? std::max<int64_t>(1, ceil_div(t, e)) : t;
  if (mode == FP8_DW) return fp8_tiles(mode, n, k, std::max<int64_t>(1, ceil_div(rows, 128)), e, !grouped, &us);
  const int64_t cols = mode == FP8_Y ? n : k, depth = mode == FP8_Y ? k : n;
  const int64_t hit = grouped ? std::min<int64_t>(e, t) : 1;   // matrices with a row, at most
  const Plan p = fp8_tiles(mode, rows, cols, ceil_div(depth, 128), std::max<int64_t>(1, hit), !grouped, &us, grouped);
  const bool few = mode == FP8_Y && rows <= 128 && hit * ceil_div(n, 16) < kMostItems;
  const double find = grouped ? std::min(fp8_idle_us(hit, e, n), fp8_search_us(hit, e, n)) : 0;
  return few && fp8_rows_us(rows, k, n, hit) + find < us ? Plan{0, 1} : p;
}

// Whether the product's launches stay below kMostItems (products by expert walk their tiles with
// a grid of the card's size).
inline bool fp8_fits(Fp8Mode mode, int64_t t, int64_t k, int64_t n, int32_t e, bool grouped) {
  if (t == 0 && mode != FP8_DW) return true;
  const Plan p = fp8_plan(mode, t, k, n, e, grouped);
  if (p.tile == 0) return true;   // (fp8_rows_grid: below kMostItems)
  if (mode == FP8_DW) return ceil_div(n, p.tile) * ceil_div(k, p.tile) * e * p.ksplit < kMostItems;
  const int64_t cols = mode == FP8_Y ? n : k;
  return ((grouped ? t / p.tile + e : ceil_div(t, p.tile))) * ceil_div(cols, p.tile) * p.ksplit < (grouped ? int64_t(1) << 31 : kMostItems);
}

}  // namespace q4
