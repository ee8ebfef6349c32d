// Launchers of the e4m3 products with a scale per block of 128 (fp8.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace q4 {

// Codes and scales of x [t][k] (gated: of silu(g) u, x [t][2 k] = g | u), each where its pointer is
// given: along the row, q_row [t][k] and s_row [k / 128][t]; along the tokens, q_col [t][k] and
// s_col [groups][k], the groups of 128 rows starting anew at each offsets[x] (offsets NULL: at row 0).
// Rows from offsets[e] on are left out.
struct Fp8QuantArgs {
  const void* x;
  int64_t t, k;
  int32_t dtype, gated;
  uint8_t *q_row, *q_col;
  float *s_row, *s_col;
  const int32_t* offsets;
  int32_t e;
};
hipError_t launch_quantize_fp8_tokens(const Fp8QuantArgs& a, hipStream_t st);
// Codes of e matrices w [e][n][k] by blocks of 128 x 128: q [e][n][k], s [e][n / 128][k / 128].
hipError_t launch_quantize_fp8_blocks(const void* w, int dtype, int64_t e, int64_t n, int64_t k, uint8_t* q, float* s,
                                      hipStream_t st);

// y[t][n] = sum_g s[g][t] ws[n / 128][g] sum_{k in g} q[t][k] wq[n][k]; rows offsets[x] .. of matrix x.
int64_t fp8_linear_workspace(int64_t t, int64_t k, int64_t n, int32_t e, bool grouped);
hipError_t launch_fp8_linear(const uint8_t* q, const float* s, int64_t t, int64_t k, const uint8_t* wq, const float* ws,
                             int64_t n, const int32_t* offsets, int32_t e, int y_dtype, void* y, void* work,
                             hipStream_t st);
// dx = codes(dy) W and dw = column codes(dy)^T (column codes of x).
int64_t fp8_linear_bwd_workspace(int64_t t, int64_t k, int64_t n, int32_t e, bool grouped);
hipError_t launch_fp8_linear_bwd(const void* dy, int64_t t, int64_t k, int64_t n, int dtype, const uint8_t* xq,
                                 const float* xs, const uint8_t* wq, const float* ws, const int32_t* offsets, int32_t e,
                                 void* dx, void* dw, void* work, hipStream_t st);

}  // namespace q4
