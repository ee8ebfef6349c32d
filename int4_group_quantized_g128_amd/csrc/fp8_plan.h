// Which kernel, tile and K split an e4m3 product takes (host arithmetic on its sizes alone).
#pragma once
#include "dense_plan.h"

namespace q4 {

// y = x W^T; dx = dy W; dW = dy^T x.
enum Fp8Mode { FP8_Y = 0, FP8_DX = 1, FP8_DW = 2 };

// A launch holds fewer workgroups than this (of up to 512 threads: below 2^32 in all).
constexpr int64_t kMostItems = int64_t(1) << 23;

// Square tiles of `bm`, K in `ks` slices of whole 128-element steps: the estimate of plan_us with
// these products' step times.
inline double fp8_plan_us(int64_t m, int64_t n, int64_t steps, int batches, int bm, int64_t ks) {
  const int t = bm == 64 ? 0 : bm == 128 ? 1 : 2;
  static const int held[3] = {3, 2, 1};
  static const double alone[3] = {0.40, 0.80, 1.40}, full[3] = {0.25, 0.45, 1.40}, ends[3] = {2.0, 4.0, 8.0};
  const int64_t per = ceil_div(steps, ks);
  const int64_t wgs = ceil_div(m, bm) * ceil_div(n, bm) * batches * ceil_div(steps, per);
  if (wgs >= kMostItems || (ks > 1 && m * ceil_div(n, 4) >= int64_t(1) << 32)) return 1e300;
  const int64_t rounds = ceil_div(wgs, 256 * held[t]);
  const int64_t last = std::min<int64_t>(held[t], ceil_div(wgs - (rounds - 1) * 256 * held[t], 256));
  const auto slice = [&](int64_t on_cu) { return ends[t] + per * std::max(alone[t], full[t] * on_cu); };
  double us = (rounds - 1) * slice(held[t]) + slice(last);
  if (ks > 1) us += 2.9 + 0.5 * ks + double(ks) * m * n * 4 / 4.5e6;
  return us;
}

inline Plan fp8_tiles(int64_t m, int64_t n, int64_t steps, int batches, bool split) {
  Plan best{64, 1};
  double us = 1e301;
  for (const int bm : {64, 128, 256})
    for (const int ks : {1, 2, 3, 4, 6, 8, 12, 16}) {
      if (ks > 1 && (!split || steps / ks < 2)) break;
      const double u = fp8_plan_us(m, n, steps, batches, bm, ks);
      if (u < us) us = u, best = Plan{bm, int(ceil_div(steps, ceil_div(steps, ks)))};
    }
  return best;
}

// The product over t rows in all, e matrices of them with `grouped`.
inline Plan fp8_plan(Fp8Mode mode, int64_t t, int64_t k, int64_t n, int32_t e, bool grouped) {
  if (mode == FP8_DW) return fp8_tiles(n, k, std::max<int64_t>(1, ceil_div(ceil_div(t, e), 128)), e, !grouped);
  const int64_t cols = mode == FP8_Y ? n : k, depth = mode == FP8_Y ? k : n;
  if (!grouped) {
    if (mode == FP8_Y && t <= 16) return Plan{0, 1};
    return fp8_tiles(t, cols, ceil_div(depth, 128), 1, true);
  }
  const int64_t rows = ceil_div(t, e);
  if (mode == FP8_Y && rows <= 32 && e * ceil_div(n, 16) < kMostItems) return Plan{0, 1};
  return Plan{rows <= 64 ? 64 : rows <= 256 ? 128 : 256, 1};
}

// Whether the product's launches stay below kMostItems (products by expert walk their tiles with
// a grid of the card's size).
inline bool fp8_fits(Fp8Mode mode, int64_t t, int64_t k, int64_t n, int32_t e, bool grouped) {
  if (t == 0 && mode != FP8_DW) return true;
  const Plan p = fp8_plan(mode, t, k, n, e, grouped);
  if (p.tile == 0) return ceil_div(n, 16) * e < kMostItems;
  if (mode == FP8_DW) return ceil_div(n, p.tile) * ceil_div(k, p.tile) * e * p.ksplit < kMostItems;
  const int64_t cols = mode == FP8_Y ? n : k;
  return ((grouped ? t / p.tile + e : ceil_div(t, p.tile))) * ceil_div(cols, p.tile) * p.ksplit < (grouped ? int64_t(1) << 31 : kMostItems);
}

}  // namespace q4
