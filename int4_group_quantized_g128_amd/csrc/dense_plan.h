// Which kernel, tile and K split a dense product takes (host arithmetic on its sizes alone).
#pragma once
#include <algorithm>
#include <cstdint>

namespace q4 {

struct Plan {
  int tile, ksplit;   // tile 0: the few-rows kernel
};

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The products by how their panels lie, which decides what a step costs.
enum Kind { NT = 0 /* forward, KC x KC */, DX = 1 /* KC x MC */, DW = 2 /* MC x MC */ };

// Estimated time (us) of a product of `steps` 128-byte K steps with square tiles of `bm` and
// K in `ks` slices.  Per kind and tile size: time of a step when the workgroup is alone on
// its CU (a chain of copy, LDS and matrix-core latencies) and when the CU is full (per
// workgroup), time of a workgroup's start and end.  They were fitted to 75 forward shapes (17
// to 2048 rows, K 512 to 16384) and 6 backward ones with an earlier end of a tile and rank plans
// rather than predict times: the estimate leaves out the results' bytes (gated 4096 x 2048 x
// 8192 with g and u 173 us against 274 measured, INT8 333 x 1040 x 1001 4.3 against 8.1).
// Today's kernels, each of the three tiles with K in 1, 2, 4 and 8 slices against the plan: of 76
// forward shapes (24 to 4096 rows, with and without g and u) 72 within 8 % of the fastest, the
// worst INT8 333 x 7168 x 7168 (44 us, 64 / 1 36) and gated 2048 x 512 x 1408 with g and u (22.5,
// 128 / 1 17); of 20 backward passes 19 within 5 %, the worst 2048 x 1000 x 2728 (105, dx by
// 128 / 2 95).  (A rule that only counted workgroups lost up to 70 %.)
inline double plan_us(Kind kind, int64_t m, int64_t n, int panels, int64_t steps, int batches, int bm, int64_t ks) {
  const int t = bm == 64 ? 0 : bm == 128 ? 1 : 2;
  static const int held[3] = {3, 2, 1};   // workgroups a CU holds
  static const double alone[3][3] = {{0.27, 0.55, 0.62}, {0.35, 0.66, 1.27}, {0.17, 0.39, 1.53}};
  static const double full[3][3] = {{0.21, 0.45, 1.23}, {0.22, 0.65, 1.27}, {0.20, 0.54, 1.53}};
  static const double ends[3][3] = {{1.9, 8.0, 4.0}, {2.9, 5.1, 13.5}, {2.0, 4.1, 9.3}};
  const int64_t per = ceil_div(steps, ks);
  const int64_t wgs = ceil_div(m, bm) * ceil_div(n * panels, bm) * batches * ceil_div(steps, per);
  // the grid stays below 2^31 workgroups, a join below 2^32 threads
  if (wgs >= int64_t(1) << 31 || (ks > 1 && m * batches * ceil_div(n, 4) >= int64_t(1) << 32)) return 1e300;
  const int64_t rounds = ceil_div(wgs, 256 * held[t]);
  const int64_t last = std::min<int64_t>(held[t], ceil_div(wgs - (rounds - 1) * 256 * held[t], 256));
  const auto slice = [&](int64_t on_cu) {
    return ends[kind][t] + per * std::max(alone[kind][t], full[kind][t] * on_cu);
  };
  double us = (rounds - 1) * slice(held[t]) + slice(last);
  // the join: a launch, a chain of reads, and the slices' bytes at 4.5 TB/s
  if (ks > 1) us += 2.9 + 0.5 * ks + double(ks) * m * n * panels * batches * 4 / 4.5e6;
  return us;
}

// Tile and K split with the least estimated time.
inline Plan plan_of(Kind kind, int64_t m, int64_t n, int panels, int64_t steps, int batches) {
  Plan best{64, 1};
  if (steps == 0) return best;   // no tokens: the weight gradients are zero
  double us = plan_us(kind, m, n, panels, steps, batches, 64, 1);
  for (const int bm : {64, 128, 256})
    for (const int ks : {1, 2, 3, 4, 6, 8, 12, 16}) {
      if (ks > 1 && steps / ks < 2) break;
      const double u = plan_us(kind, m, n, panels, steps, batches, bm, ks);
      if (u < us) us = u, best = Plan{bm, int(ceil_div(steps, ceil_div(steps, ks)))};
    }
  return best;
}

// The few-rows kernel up to 16 rows (16 rows, gated 2048 / 2048: 6.4 us against 10.1 in tiles;
// INT8 8192 x 2048: 9.6 against 10.9), but tiles from 8 rows on where the columns fill the chip
// with them, since they read x once per 64 columns and not per 8 or 16 (gated 7168 / 7168, 8
// rows: 50.2 against 41.2 us, 16 rows: 56.5 against 41.8; 2048 / 8192, 16 rows: 16.2 / 15.4).
// cols: columns of all B panels.
inline bool few_rows(int64_t t, int64_t cols) { return t < 8 || (t <= 16 && ceil_div(cols, 64) < 224); }

// The products of the INT8 linear, the gated projection and its gradients (tokens > 0).
inline Plan int8_plan(int64_t t, int64_t k, int64_t n) {
  return few_rows(t, n) ? Plan{0, 1} : plan_of(NT, t, n, 1, ceil_div(k, 128), 1);
}
inline Plan swiglu_plan(int64_t t, int64_t h, int64_t i) {
  return few_rows(t, 2 * i) ? Plan{0, 1} : plan_of(NT, t, i, 2, ceil_div(h, 64), 1);
}
inline Plan dx_plan(int64_t t, int64_t h, int64_t i) { return plan_of(DX, t, h, 1, 2 * ceil_div(i, 64), 1); }
inline Plan dw_plan(int64_t t, int64_t h, int64_t i) { return plan_of(DW, i, h, 1, ceil_div(t, 64), 2); }

}  // namespace q4
