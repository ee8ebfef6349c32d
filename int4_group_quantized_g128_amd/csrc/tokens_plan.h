// Which workgroups sort tokens by expert (host arithmetic on the sizes alone).
#pragma once
#include <cstdint>

namespace q4 {

// Whether a token's row, of row_bytes, goes out by a wave, four tokens a workgroup, rather than by a
// workgroup: where it is narrow, or not wide and goes to few places (4096 tokens of 2048, k = 2: 27.2
// -> 24.0 us with the order, as codes 25.0 -> 23.2; of 1024, k = 4, 26.2 -> 24.5 and 24.0 -> 21.0), and
// the tokens are at least seven workgroups for each of 256 CUs: each of a workgroup's tokens is ranked
// by all of its waves before the first row goes out (rows / codes, 16 tokens of 256, k = 8: 6.4 / 7.0 us by
// workgroups, 12.7 / 13.1 by waves; 300 of 512, k = 8, 12.3 / 12.9 and 17.4 / 17.8; 1500 of 2048, k = 2,
// 14.5 / 14.6 and 15.3 / 17.2; 2000 of 256, k = 2, 14.1 / 14.6 and 12.4 / 12.8).
inline bool dispatch_by_waves(int64_t t, int32_t k, int64_t row_bytes) {
  return t >= 7 * 256 && k <= 64 && row_bytes <= (k <= 4 ? 4096 : 1024);
}

}  // namespace q4
