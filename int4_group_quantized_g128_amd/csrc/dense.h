// Launchers of the dense operators around the quantised FFN (dense.hip, norm.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace q4 {

// Norms around a block (norm.hip).  dtype as Q4_F32 / Q4_F16 / Q4_BF16.
enum GateKind { kGateNone = 0, kGateChannel = 1, kGateToken = 2, kGateElement = 3 };
struct BlockNormArgs {
  int64_t rows;
  int32_t cols;
  int32_t gate_kind;
  float alpha;
  float eps;
  const void* res;
  const void* y;       // NULL: r = res
  const void* w_post;  // NULL: p = y
  const void* gate;
  const void* w_pre;   // NULL: no n
};
int block_norm_max_cols();
hipError_t launch_block_norm(const BlockNormArgs& a, int dtype, void* r_out, void* n_out, int8_t* q_out, float* s_out,
                             hipStream_t st);
int64_t block_norm_bwd_workspace(int64_t rows, int64_t cols);
hipError_t launch_block_norm_bwd(const BlockNormArgs& a, int dtype, const void* dr, const void* dn, void* dres,
                                 void* dy, float* dw_post, void* dgate, float* dw_pre, float* partial,
                                 hipStream_t st);

// Dense products (dense.hip).
// INT8 weight rows: s = amax / 127, q = clamp(rint(w / s), -127, 127).
hipError_t launch_quantize8_rows(const void* w, int dtype, int64_t n, int64_t k, int8_t* q, float* s, int32_t* flags,
                                 hipStream_t st);
// y[t][n] = (q w_q^T) * (s[t] * w_s[n]) (+ bias[n]); y_dtype as Q4_F32 / Q4_F16 / Q4_BF16.
int64_t int8_linear_workspace(int64_t t, int64_t k, int64_t n);
hipError_t launch_int8_linear(const int8_t* q, const float* s, int64_t t, int64_t k, const int8_t* wq, const float* ws,
                              int64_t n, const float* bias, int y_dtype, void* y, void* work, hipStream_t st);
// h = silu(x wg^T) * (x wu^T); gu (optional) fp32 [t][2][i] the two products.  f16: fp16, else bf16.
int64_t swiglu_linear_workspace(int64_t t, int64_t h, int64_t i);
hipError_t launch_swiglu_linear(const void* x, const void* wg, const void* wu, int64_t t, int64_t h, int64_t i, int f16,
                                void* out, float* gu, void* work, hipStream_t st);
int64_t swiglu_linear_bwd_workspace(int64_t t, int64_t h, int64_t i);
hipError_t launch_swiglu_linear_bwd(const void* dh, const void* x, const void* wg, const void* wu, const float* gu,
                                    int64_t t, int64_t h, int64_t i, int f16, void* dx, void* dwg, void* dwu,
                                    void* work, hipStream_t st);

}  // namespace q4
