// Norms before and after a block, fused with the block's gate and residual scale
// (forward and backward).
//
//   p = N(y; w_post)  (or y),  r = res + alpha * gate * p,  n = N(r; w_pre),
//   N(v; w)_i = v_i * rstd(v) * w_i,  rstd(v) = 1 / sqrt(mean(v^2) + eps).
//
// Backward, with vh = v * rstd(v) and
//   D(v; w, d) = rstd * (w d - vh * mean(w d vh))        (gradient of N to v):
//   dr'   = dr + D(r; w_pre, dn)          dw_pre  = sum_rows dn * rh
//   dres  = dr',  e = alpha * dr'         dgate   = sum over the gate's broadcast axis of e * p
//   dp    = e * gate                      dw_post = sum_rows dp * yh
//   dy    = D(y; w_post, dp)              (dp without w_post)
//
// Bound by memory: a row is read once, kept in registers through every reduction and
// written once; the row statistics are recomputed in the backward pass from the rows it
// reads anyway, so nothing but the inputs is kept between the passes.  All sums are fp32;
// n and the gradients are formed from the unrounded r, and each output is rounded once.
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "dense.h"

namespace q4 {

namespace {

constexpr int kMaxCols = 16384;
constexpr int kBwdWaves = 8;
constexpr int kGradSlots = 3;   // partial sums per workgroup: dw_pre, dw_post, channel gate

struct NF32 {};
struct NF16 {};
struct NBF16 {};
template <typename T> struct Elem;
template <> struct Elem<NF32> {
  typedef float type;
  static Q4_DEVICE float up(float v) { return v; }
  static Q4_DEVICE float down(float v) { return v; }
};
template <> struct Elem<NF16> {
  typedef uint16_t type;
  static Q4_DEVICE float up(uint16_t v) { return f16_bits_to_f32(v); }
  static Q4_DEVICE uint16_t down(float v) { return bitcast<uint16_t>(_Float16(v)); }
};
template <> struct Elem<NBF16> {
  typedef uint16_t type;
  static Q4_DEVICE float up(uint16_t v) { return bf16_to_f32(v); }
  static Q4_DEVICE uint16_t down(float v) { return bitcast<uint16_t>(__bf16(v)); }
};

// Columns of thread `tid` of TPR threads that share a row: NV vectors of 8 consecutive
// columns, vector j at 8 (j TPR + tid) (VEC: 16-byte accesses, cols % 8 == 0), or NV * 8
// single columns e TPR + tid.
template <typename T, int TPR, int NV, bool VEC>
struct Row {
  typedef typename Elem<T>::type S;
  static constexpr int N = NV * 8;

  // The thread's part of a row as stored (16-byte registers, or one value each).
  struct Raw {
    static constexpr int Q = VEC ? NV * int(sizeof(S)) / 2 : 1;
    uint4 q[Q];
    S e[VEC ? 1 : N];
  };
  static Q4_DEVICE Raw fetch(const void* base, int64_t row, int cols, int tid) {
    const S* p = static_cast<const S*>(base) + row * cols;
    Raw r;
    if constexpr (VEC) {
      constexpr int PER = sizeof(S) / 2;   // 16-byte registers per vector
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = 8 * (j * TPR + tid);
#pragma unroll
        for (int h = 0; h < PER; ++h) r.q[j * PER + h] = c < cols ? load16(p + c + 4 * h) : make_uint4(0, 0, 0, 0);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = i * TPR + tid;
        r.e[i] = c < cols ? p[c] : S(0);
      }
    }
    return r;
  }
  // Every element the same value (a missing weight is ones, a token's gate its value).
  static Q4_DEVICE Raw fill(S v) {
    Raw r;
    uint32_t u;
    if constexpr (sizeof(S) == 4) u = __float_as_uint(v);
    else u = v | uint32_t(v) << 16;
#pragma unroll
    for (int j = 0; j < Raw::Q; ++j) r.q[j] = make_uint4(u, u, u, u);
#pragma unroll
    for (int i = 0; i < (VEC ? 1 : N); ++i) r.e[i] = v;
    return r;
  }
  static Q4_DEVICE float at(const Raw& r, int i) {
    if constexpr (!VEC) {
      return Elem<T>::up(r.e[i]);
    } else if constexpr (sizeof(S) == 4) {
      const uint4 v = r.q[i / 4];
      return __uint_as_float(i % 4 == 0 ? v.x : i % 4 == 1 ? v.y : i % 4 == 2 ? v.z : v.w);
    } else {
      const uint4 v = r.q[i / 8];
      const int w = i % 8 / 2;
      const uint32_t u = w == 0 ? v.x : w == 1 ? v.y : w == 2 ? v.z : v.w;
      return Elem<T>::up(S(i % 2 ? u >> 16 : u & 0xffffu));
    }
  }

  static Q4_DEVICE void store(void* base, int64_t row, int cols, int tid, const float v[N]) {
    S* p = static_cast<S*>(base) + row * cols;
    if constexpr (VEC) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = 8 * (j * TPR + tid);
        if (c < cols) {
          S t[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) t[i] = Elem<T>::down(v[8 * j + i]);
          *reinterpret_cast<uint4*>(p + c) = *reinterpret_cast<const uint4*>(t);
          if constexpr (sizeof(S) == 4)
            *reinterpret_cast<uint4*>(p + c + 4) = *reinterpret_cast<const uint4*>(t + 4);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = i * TPR + tid;
        if (c < cols) p[c] = Elem<T>::down(v[i]);
      }
    }
  }

  static Q4_DEVICE void store_f32(float* p, int cols, int tid, const float v[N]) {
    if constexpr (VEC) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = 8 * (j * TPR + tid);
        if (c < cols) {
          *reinterpret_cast<f32x4_t*>(p + c) = f32x4_t{v[8 * j], v[8 * j + 1], v[8 * j + 2], v[8 * j + 3]};
          *reinterpret_cast<f32x4_t*>(p + c + 4) = f32x4_t{v[8 * j + 4], v[8 * j + 5], v[8 * j + 6], v[8 * j + 7]};
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = i * TPR + tid;
        if (c < cols) p[c] = v[i];
      }
    }
  }

  static Q4_DEVICE void store_codes(int8_t* base, int64_t row, int cols, int tid, const float v[N]) {
    int8_t* p = base + row * cols;
    if constexpr (VEC) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = 8 * (j * TPR + tid);
        if (c < cols) {
          int8_t t[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) t[i] = int8_t(int(v[8 * j + i]));
          *reinterpret_cast<uint2*>(p + c) = *reinterpret_cast<const uint2*>(t);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = i * TPR + tid;
        if (c < cols) p[c] = int8_t(int(v[i]));
      }
    }
  }
};

// Sum (or maximum) of K values over the WPR waves of a row.  `slots` holds one float per
// (use, value, wave of the workgroup); consecutive uses alternate between two halves, so
// one barrier per reduction is enough.
template <int WPR, int K, bool MAX = false>
Q4_DEVICE void row_reduce(float v[K], float* slots, int wave, int& phase) {
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
      const float other = __shfl_xor(v[k], o, 64);
      v[k] = MAX ? fmaxf(v[k], other) : v[k] + other;
    }
  if constexpr (WPR > 1) {
    float* s = slots + phase * 2 * 16;
    phase ^= 1;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) s[k * 16 + wave] = v[k];
    __syncthreads();
    const int first = wave / WPR * WPR;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float a = s[k * 16 + first];
#pragma unroll
      for (int w = 1; w < WPR; ++w) a = MAX ? fmaxf(a, s[k * 16 + first + w]) : a + s[k * 16 + first + w];
      v[k] = a;
    }
  }
}

Q4_DEVICE float rstd_of(float sumsq, int cols, float eps) { return 1.0f / sqrtf(sumsq / float(cols) + eps); }

// Rows of a workgroup at a time: one, or four where a row is one wave's (no barriers).
template <int WPR> constexpr int rows_per_wg() { return WPR == 1 ? 4 : 1; }
template <int WPR> constexpr int threads_per_wg() { return 64 * WPR * rows_per_wg<WPR>(); }

// Whether the next row is fetched ahead (16 waves of 128 registers, or single columns, have
// no room for it).
template <int WPR, bool VEC> constexpr bool fetch_ahead() { return VEC && WPR < 16; }

// Every workgroup walks rows base, base + step, ...: the weights stay in its registers, and
// the next row is on its way while the current one is reduced.  16-bit rows of vectors run four
// waves per SIMD (4096 x 7168 bf16 with a channel gate: two workgroups per CU, 41 us, 5.7 TB/s);
// fp32 ones two or three, without loss (4096 x 7168 95 us, 4.9 TB/s).  Single columns are bound by
// their accesses of one element: 4096 x 7167 bf16 121 us.
template <typename T, int WPR, int NV, bool VEC>
__global__ void __launch_bounds__(threads_per_wg<WPR>()) __attribute__((amdgpu_waves_per_eu(sizeof(typename Elem<T>::type) == 2 && VEC ? 4 : 1))) k_block_norm_fwd(BlockNormArgs a, void* r_out, void* n_out,
                                                                          int8_t* q_out, float* s_out) {
  typedef Row<T, 64 * WPR, NV, VEC> R;
  typedef typename R::Raw Raw;
  constexpr int N = R::N;
  __shared__ float slots[2 * 2 * 16];
  const int wave = threadIdx.x >> 6;
  const int tid = threadIdx.x % (64 * WPR);
  const int cols = a.cols;
  int phase = 0;
  const int64_t step = int64_t(gridDim.x) * rows_per_wg<WPR>();
  int64_t row = int64_t(blockIdx.x) * rows_per_wg<WPR>() + threadIdx.x / (64 * WPR);
  if (row >= a.rows) return;   // whole waves, and with WPR > 1 the whole workgroup
  const Raw ones = R::fill(Elem<T>::down(1.f));
  Raw w_post = ones, w_pre = ones, gate = ones, res = ones, y = ones;
  if (a.w_post) w_post = R::fetch(a.w_post, 0, cols, tid);
  if (a.w_pre) w_pre = R::fetch(a.w_pre, 0, cols, tid);
  if (a.gate_kind == kGateChannel) gate = R::fetch(a.gate, 0, cols, tid);
  auto fetch = [&](int64_t row, Raw& res, Raw& y, Raw& gate) {
    res = R::fetch(a.res, row, cols, tid);
    if (a.y) y = R::fetch(a.y, row, cols, tid);
    if (a.gate_kind == kGateElement) gate = R::fetch(a.gate, row, cols, tid);
    if (a.gate_kind == kGateToken) gate = R::fill(static_cast<const typename R::S*>(a.gate)[row]);
  };
  constexpr bool AHEAD = fetch_ahead<WPR, VEC>();
  if constexpr (AHEAD) fetch(row, res, y, gate);
  for (; row < a.rows; row += step) {
    Raw next_res, next_y, next_gate;
    if constexpr (AHEAD) {
      next_res = res, next_y = y, next_gate = gate;
      if (row + step < a.rows) fetch(row + step, next_res, next_y, next_gate);
    } else {
      fetch(row, res, y, gate);
    }
    float r[N];
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = R::at(res, i);
    if (a.y) {
      float rs = 1.f;
      if (a.w_post) {
        float ss[1] = {0.f};
#pragma unroll
        for (int i = 0; i < N; ++i) ss[0] += R::at(y, i) * R::at(y, i);
        row_reduce<WPR, 1>(ss, slots, wave, phase);
        rs = rstd_of(ss[0], cols, a.eps);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) r[i] += a.alpha * (R::at(gate, i) * (R::at(y, i) * rs * R::at(w_post, i)));
      R::store(r_out, row, cols, tid, r);
    }
    if (a.w_pre) {
      float ss[1] = {0.f};
#pragma unroll
      for (int i = 0; i < N; ++i) ss[0] += r[i] * r[i];
      row_reduce<WPR, 1>(ss, slots, wave, phase);
      const float rs = rstd_of(ss[0], cols, a.eps);
#pragma unroll
      for (int i = 0; i < N; ++i) r[i] = r[i] * rs * R::at(w_pre, i);
      if (q_out) {
        // per-token INT8 codes of the unrounded n, by the rule of act_quant_int8
        // (a row with a NaN or an infinity, which no code holds, gets codes 0 and a NaN scale)
        float mx[1] = {0.f};
#pragma unroll
        for (int i = 0; i < N; ++i) mx[0] = fmaxf(mx[0], r[i] != r[i] ? __builtin_inff() : fabsf(r[i]));
        row_reduce<WPR, 1, true>(mx, slots, wave, phase);
        const bool finite = mx[0] < __builtin_inff();
        const float s = mx[0] / 127.0f;
#pragma unroll
        for (int i = 0; i < N; ++i)
          r[i] = finite && s > 0.f ? fminf(fmaxf(rintf(r[i] / s), -128.f), 127.f) : 0.f;
        R::store_codes(q_out, row, cols, tid, r);
        if (tid == 0) s_out[row] = finite ? s : __builtin_nanf("");
      } else {
        R::store(n_out, row, cols, tid, r);
      }
    }
    if constexpr (AHEAD) res = next_res, y = next_y, gate = next_gate;
  }
}

// As the forward kernel; the contributions to the weight (and channel gate) gradients are
// added in registers, and partial [workgroups][3][cols] gets one set per workgroup, which
// k_norm_grad_sum adds in order.  One kernel for every combination of parts: up to 8192 columns
// in 16 bits its 250 registers hold (4096 x 7168 bf16 85 us in all, 4.1 TB/s), fp32 rows of up
// to 4096 take 297 (one wave per SIMD; 4096 x 4096 93 us, 4.3 TB/s).  Beyond that it spills:
// fp32 rows of 4104 to 8192 columns 1140 bytes per lane (4096 x 7168 1680 us), rows above 8192
// 336 to 460 in every type (2048 x 16384 bf16 383 us).
template <typename T, int WPR, int NV, bool VEC>
__global__ void __launch_bounds__(threads_per_wg<WPR>())
    k_block_norm_bwd(BlockNormArgs a, const void* dr, const void* dn, void* dres, void* dy, void* dgate,
                     float* partial) {
  typedef Row<T, 64 * WPR, NV, VEC> R;
  typedef typename R::Raw Raw;
  constexpr int N = R::N;
  __shared__ float slots[2 * 2 * 16];
  const int wave = threadIdx.x >> 6;
  const int tid = threadIdx.x % (64 * WPR);
  const int cols = a.cols;
  int phase = 0;
  float dw_pre[N], dw_post[N], dg_ch[N];
#pragma unroll
  for (int i = 0; i < N; ++i) dw_pre[i] = dw_post[i] = dg_ch[i] = 0.f;
  const int64_t step = int64_t(gridDim.x) * rows_per_wg<WPR>();
  const int64_t group = int64_t(blockIdx.x) * rows_per_wg<WPR>() + threadIdx.x / (64 * WPR);
  const Raw ones = R::fill(Elem<T>::down(1.f));
  Raw w_post = ones, w_pre = ones, gate = ones, res = ones, y = ones, dnv = ones, drv = R::fill(0);
  if (a.w_post) w_post = R::fetch(a.w_post, 0, cols, tid);
  if (a.w_pre) w_pre = R::fetch(a.w_pre, 0, cols, tid);
  if (a.gate_kind == kGateChannel) gate = R::fetch(a.gate, 0, cols, tid);
  auto fetch = [&](int64_t row, Raw& res, Raw& y, Raw& dnv, Raw& drv, Raw& gate) {
    res = R::fetch(a.res, row, cols, tid);
    if (a.y) y = R::fetch(a.y, row, cols, tid);
    if (a.w_pre) dnv = R::fetch(dn, row, cols, tid);
    if (dr) drv = R::fetch(dr, row, cols, tid);
    if (a.gate_kind == kGateElement) gate = R::fetch(a.gate, row, cols, tid);
    if (a.gate_kind == kGateToken) gate = R::fill(static_cast<const typename R::S*>(a.gate)[row]);
  };
  constexpr bool AHEAD = fetch_ahead<WPR, VEC>();
  if (AHEAD && group < a.rows) fetch(group, res, y, dnv, drv, gate);
  for (int64_t row = group; row < a.rows; row += step) {   // (the same trip count for a row's waves)
    Raw n_res, n_y, n_dn, n_dr, n_gate;
    if constexpr (AHEAD) {
      n_res = res, n_y = y, n_dn = dnv, n_dr = drv, n_gate = gate;
      if (row + step < a.rows) fetch(row + step, n_res, n_y, n_dn, n_dr, n_gate);
    } else {
      fetch(row, res, y, dnv, drv, gate);
    }
    float r[N], yh[N];
    float rs_y = 1.f;
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = R::at(res, i);
    if (a.y) {
      if (a.w_post) {
        float ss[1] = {0.f};
#pragma unroll
        for (int i = 0; i < N; ++i) ss[0] += R::at(y, i) * R::at(y, i);
        row_reduce<WPR, 1>(ss, slots, wave, phase);
        rs_y = rstd_of(ss[0], cols, a.eps);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        yh[i] = R::at(y, i) * rs_y;
        r[i] += a.alpha * (R::at(gate, i) * (yh[i] * R::at(w_post, i)));
      }
    }
    float d[N];
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = R::at(drv, i);   // zeros without dr
    if (a.w_pre) {
      float red[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < N; ++i) {
        red[0] += r[i] * r[i];
        red[1] += R::at(w_pre, i) * R::at(dnv, i) * r[i];
      }
      row_reduce<WPR, 2>(red, slots, wave, phase);
      const float rs = rstd_of(red[0], cols, a.eps);
      const float c = red[1] * rs / float(cols);   // mean(w dn rh)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float rh = r[i] * rs;
        d[i] += rs * (R::at(w_pre, i) * R::at(dnv, i) - rh * c);
        dw_pre[i] += R::at(dnv, i) * rh;
      }
    }
    R::store(dres, row, cols, tid, d);
    if (a.y) {
      float red[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float e = a.alpha * d[i];
        r[i] = e * (yh[i] * R::at(w_post, i));   // e p, the gate's gradient before its sum
        dg_ch[i] += r[i];
        red[1] += r[i];
        d[i] = e * R::at(gate, i);               // dp
        const float dy = d[i] * yh[i];
        dw_post[i] += dy;
        red[0] += dy * R::at(w_post, i);
      }
      if (a.gate_kind == kGateElement) R::store(dgate, row, cols, tid, r);
      if (a.w_post || a.gate_kind == kGateToken) row_reduce<WPR, 2>(red, slots, wave, phase);
      if (a.gate_kind == kGateToken && tid == 0) static_cast<float*>(dgate)[row] = red[1];
      if (a.w_post) {
        const float c = red[0] / float(cols);
#pragma unroll
        for (int i = 0; i < N; ++i) d[i] = rs_y * (d[i] * R::at(w_post, i) - yh[i] * c);
      }
      R::store(dy, row, cols, tid, d);
    }
    if constexpr (AHEAD) res = n_res, y = n_y, dnv = n_dn, drv = n_dr, gate = n_gate;
  }
  // one set of sums per workgroup: its row groups' sums join through LDS in group order
  float* out = partial + int64_t(blockIdx.x) * kGradSlots * cols;
  auto put = [&](float* to, const float v[N]) {
    if constexpr (rows_per_wg<WPR>() == 1) {
      R::store_f32(to, cols, tid, v);
    } else {
      constexpr int G = rows_per_wg<WPR>();
      __shared__ __align__(16) float sums[G][64 * WPR * N];
      R::store_f32(sums[threadIdx.x / (64 * WPR)], cols, tid, v);
      __syncthreads();
      for (int c = threadIdx.x; c < cols; c += threads_per_wg<WPR>()) {
        float acc = sums[0][c];
#pragma unroll
        for (int k = 1; k < G; ++k) acc += sums[k][c];
        to[c] = acc;
      }
      __syncthreads();
    }
  };
  if (a.w_pre) put(out, dw_pre);
  if (a.w_post) put(out + cols, dw_post);
  if (a.gate_kind == kGateChannel) put(out + 2 * cols, dg_ch);
}

// out[slot][c] = sum over the workgroups of partial[group][slot][c]: a workgroup owns 64
// columns of one slot, its 16 waves take every 16th group, and wave 0 adds the 16 sums in
// wave order (a fixed order: equal inputs give equal bits).
__global__ void __launch_bounds__(1024) k_norm_grad_sum(const float* __restrict__ partial, int groups, int cols,
                                                        float* dw_pre, float* dw_post, float* dg_ch) {
  __shared__ float s[16][64];
  float* out = blockIdx.y == 0 ? dw_pre : blockIdx.y == 1 ? dw_post : dg_ch;
  if (!out) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  float acc = 0.f;
  if (c < cols) {
    const float* p = partial + int64_t(blockIdx.y) * cols + c;
#pragma unroll 4
    for (int g = wave; g < groups; g += 16) acc += p[int64_t(g) * kGradSlots * cols];
  }
  s[wave][lane] = acc;
  __syncthreads();
  if (wave == 0 && c < cols) {
#pragma unroll
    for (int w = 1; w < 16; ++w) acc += s[w][lane];
    out[c] = acc;
  }
}

// Workgroups of a pass over the rows: 16 waves per CU in the forward pass, 8 in the backward
// one, which holds twice as much per thread and writes three partial rows of fp32 per workgroup.
// That is what a CU holds at once of 16-bit rows with two vectors per lane; of fp32 ones it holds
// 8 to 12 and 4, and the other workgroups start as these end.
int64_t pass_wgs(int64_t rows, int wpr, bool backward) {
  const int rpw = wpr == 1 ? 4 : 1;
  const int64_t fill = 256 * std::max(1, (backward ? kBwdWaves : 16) / (wpr * rpw));
  return std::min<int64_t>((rows + rpw - 1) / rpw, fill);
}

// Waves per row: two vectors of 8 columns per lane (one to 512 columns), or 8 single columns,
// which take a register each (16 of them beyond 8192).  Up to 2048 columns few rows take four
// waves of one vector each, whose chain is shorter (one row to INT8 codes: 4.0 us against 4.5), many
// rows two waves (4096 x 2048: forward 14.8 -> 13.9 us, with INT8 codes 13.4 -> 11.7).
int waves_per_row(int64_t rows, int64_t cols) {
  if (cols % 8 != 0) return cols <= 512 ? 1 : cols <= 2048 ? 4 : cols <= 4096 ? 8 : 16;
  if (cols <= 1024) return 1;
  if (cols <= 2048) return rows >= 1024 ? 2 : 4;
  return cols <= 4096 ? 4 : cols <= 8192 ? 8 : 16;
}

template <bool VEC, typename F>
hipError_t with_shape(int64_t rows, int64_t cols, F&& f) {
  typedef std::integral_constant<int, 1> one;
  typedef std::integral_constant<int, 2> two;
  typedef std::integral_constant<int, 4> four;
  typedef std::integral_constant<int, 8> eight;
  typedef std::integral_constant<int, 16> sixteen;
  const int w = waves_per_row(rows, cols);
  if constexpr (VEC) {
    if (w == 1) return cols <= 512 ? f(one{}, one{}) : f(one{}, two{});
    if (w == 4) return cols <= 2048 ? f(four{}, one{}) : f(four{}, two{});
    return w == 2 ? f(two{}, two{}) : w == 8 ? f(eight{}, two{}) : f(sixteen{}, two{});
  } else {
    if (w == 16) return cols <= 8192 ? f(sixteen{}, one{}) : f(sixteen{}, two{});
    return w == 1 ? f(one{}, one{}) : w == 4 ? f(four{}, one{}) : f(eight{}, one{});
  }
}

template <typename F>
hipError_t with_type(int dtype, int64_t rows, int64_t cols, F&& f) {
  const bool vec = cols % 8 == 0;
  auto go = [&](auto t, auto v) {
    constexpr bool VEC = decltype(v)::value;
    return with_shape<VEC>(rows, cols, [&](auto wpr, auto nv) { return f(t, v, wpr, nv); });
  };
  if (dtype == 0) return vec ? go(NF32{}, std::true_type{}) : go(NF32{}, std::false_type{});
  if (dtype == 1) return vec ? go(NF16{}, std::true_type{}) : go(NF16{}, std::false_type{});
  return vec ? go(NBF16{}, std::true_type{}) : go(NBF16{}, std::false_type{});
}

}  // namespace

int block_norm_max_cols() { return kMaxCols; }

hipError_t launch_block_norm(const BlockNormArgs& a, int dtype, void* r_out, void* n_out, int8_t* q_out, float* s_out,
                             hipStream_t st) {
  return with_type(dtype, a.rows, a.cols, [&](auto t, auto v, auto wpr, auto nv) {
    typedef decltype(t) T;
    constexpr int WPR = decltype(wpr)::value;
    const unsigned grid = unsigned(pass_wgs(a.rows, WPR, false));
    hipLaunchKernelGGL((k_block_norm_fwd<T, WPR, decltype(nv)::value, decltype(v)::value>), dim3(grid),
                       dim3(threads_per_wg<WPR>()), 0, st, a, r_out, n_out, q_out, s_out);
    return hipGetLastError();
  });
}

int64_t block_norm_bwd_workspace(int64_t rows, int64_t cols) {
  return pass_wgs(rows, waves_per_row(rows, cols), true) * kGradSlots * cols * 4;
}

hipError_t launch_block_norm_bwd(const BlockNormArgs& a, int dtype, const void* dr, const void* dn, void* dres,
                                 void* dy, float* dw_post, void* dgate, float* dw_pre, float* partial,
                                 hipStream_t st) {
  int groups = 0;
  if (a.rows > 0) {
    const hipError_t e = with_type(dtype, a.rows, a.cols, [&](auto t, auto v, auto wpr, auto nv) {
      typedef decltype(t) T;
      constexpr int WPR = decltype(wpr)::value;
      const int64_t wgs = pass_wgs(a.rows, WPR, true);
      groups = int(wgs);
      hipLaunchKernelGGL((k_block_norm_bwd<T, WPR, decltype(nv)::value, decltype(v)::value>), dim3(unsigned(wgs)),
                         dim3(threads_per_wg<WPR>()), 0, st, a, dr, dn, dres, dy, dgate, partial);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
  }
  float* dg_ch = a.gate_kind == kGateChannel ? static_cast<float*>(dgate) : nullptr;
  if (!dw_pre && !dw_post && !dg_ch) return hipSuccess;
  hipLaunchKernelGGL(k_norm_grad_sum, dim3(unsigned((a.cols + 63) / 64), kGradSlots), dim3(1024), 0, st, partial, groups,
                     a.cols, dw_pre, dw_post, dg_ch);
  return hipGetLastError();
}

}  // namespace q4
