// Launchers of the token order (tokens.hip): tokens sorted by expert and back.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace q4 {

// Sorts the t * k slots by expert (ids - first in [0, e); others are dropped: inv -1, perm -1
// behind the last held position) and writes the tokens' rows in that order, as they are (out:
// rows of h elements of dtype) or as e4m3 codes with a scale per 128 columns (q, s [h / 128][t k]).
struct DispatchArgs {
  const void* x;
  const int32_t* ids;
  int64_t t, h;
  int32_t k, first, e, dtype;
  void* out;
  uint8_t* q;
  float* s;
  int32_t *offsets, *perm, *inv;
};
int64_t dispatch_workspace(int64_t t, int32_t k, int32_t e);
hipError_t launch_dispatch(const DispatchArgs& a, void* work, hipStream_t st);

// out[t] = sum_j w[t][j] y[inv[t][j]] (+ add[t]); w NULL: ones; add NULL: nothing.
hipError_t launch_tokens_combine(const void* y, const int32_t* inv, const float* w, const void* add, int64_t t,
                                 int32_t k, int64_t h, int dtype, void* out, hipStream_t st);
// dy[inv[t][j]] = w[t][j] dout[t];  dw[t][j] = <dout[t], y[inv[t][j]]> (dw NULL: y is not read).
hipError_t launch_tokens_combine_bwd(const void* dout, const void* y, const int32_t* inv, const float* w, int64_t t,
                                     int32_t k, int64_t h, int dtype, void* dy, float* dw, hipStream_t st);

}  // namespace q4
