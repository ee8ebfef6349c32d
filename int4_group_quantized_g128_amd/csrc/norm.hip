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
#include <type_traits>

#include "common.h"
#include "internal.h"

namespace q4 {

namespace {

constexpr int kMaxCols = 16384;
constexpr int kGradSlots = 3;   // partial sums per row group: dw_pre, dw_post, channel gate

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
  static Q4_DEVICE uint16_t down(float v) { return f32_to_bf16(v); }
};

// Columns of thread `tid` of TPR threads that share a row: NV vectors of 8 consecutive
// columns, vector j at 8 (j TPR + tid) (VEC: 16-byte accesses, cols % 8 == 0), or NV * 8
// single columns e TPR + tid.
template <typename T, int TPR, int NV, bool VEC>
struct Row {
  typedef typename Elem<T>::type S;
  static constexpr int N = NV * 8;
  static Q4_DEVICE int col(int tid, int i) { return VEC ? 8 * ((i / 8) * TPR + tid) + i % 8 : i * TPR + tid; }

  static Q4_DEVICE void load(const void* base, int64_t row, int cols, int tid, float v[N]) {
    const S* p = static_cast<const S*>(base) + row * cols;
    if constexpr (VEC) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = 8 * (j * TPR + tid);
        if (c < cols) {
          S t[8];
          *reinterpret_cast<uint4*>(t) = load16(p + c);
          if constexpr (sizeof(S) == 4) *reinterpret_cast<uint4*>(t + 4) = load16(p + c + 4);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[8 * j + i] = Elem<T>::up(t[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[8 * j + i] = 0.f;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = i * TPR + tid;
        v[i] = c < cols ? Elem<T>::up(p[c]) : 0.f;
      }
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
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = col(tid, i);
      if (c < cols) p[c] = v[i];
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

// Rows per workgroup: four waves' worth of row groups, or one row over WPR > 4 waves.
template <int WPR> constexpr int rows_per_wg() { return WPR >= 4 ? 1 : 4 / WPR; }
template <int WPR> constexpr int threads_per_wg() { return 64 * WPR * rows_per_wg<WPR>(); }

template <typename T, int WPR, int NV, bool VEC>
__global__ void __launch_bounds__(threads_per_wg<WPR>()) k_block_norm_fwd(BlockNormArgs a, void* r_out, void* n_out,
                                                                          int8_t* q_out, float* s_out) {
  typedef Row<T, 64 * WPR, NV, VEC> R;
  constexpr int N = R::N;
  __shared__ float slots[2 * 2 * 16];
  const int wave = threadIdx.x >> 6;
  const int tid = threadIdx.x % (64 * WPR);
  const int cols = a.cols;
  int phase = 0;
  const int64_t step = int64_t(gridDim.x) * rows_per_wg<WPR>();
  for (int64_t base = int64_t(blockIdx.x) * rows_per_wg<WPR>(); base < a.rows; base += step) {
    int64_t row = base + threadIdx.x / (64 * WPR);
    if constexpr (rows_per_wg<WPR>() > 1)
      if (row >= a.rows) break;   // WPR < 4: no barrier below (WPR == 1)
    float r[N];
    R::load(a.res, row, cols, tid, r);
    if (a.y) {
      float p[N];
      R::load(a.y, row, cols, tid, p);
      if (a.w_post) {
        float w[N], ss[1] = {0.f};
        R::load(a.w_post, 0, cols, tid, w);
#pragma unroll
        for (int i = 0; i < N; ++i) ss[0] += p[i] * p[i];
        row_reduce<WPR, 1>(ss, slots, wave, phase);
        const float rs = rstd_of(ss[0], cols, a.eps);
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] = p[i] * rs * w[i];
      }
      if (a.gate_kind == kGateToken) {
        const float g = a.alpha * Elem<T>::up(static_cast<const typename R::S*>(a.gate)[row]);
#pragma unroll
        for (int i = 0; i < N; ++i) r[i] += g * p[i];
      } else if (a.gate_kind == kGateNone) {
#pragma unroll
        for (int i = 0; i < N; ++i) r[i] += a.alpha * p[i];
      } else {
        float g[N];
        R::load(a.gate, a.gate_kind == kGateElement ? row : 0, cols, tid, g);
#pragma unroll
        for (int i = 0; i < N; ++i) r[i] += a.alpha * (g[i] * p[i]);
      }
      R::store(r_out, row, cols, tid, r);
    }
    if (a.w_pre) {
      float w[N], ss[1] = {0.f};
      R::load(a.w_pre, 0, cols, tid, w);
#pragma unroll
      for (int i = 0; i < N; ++i) ss[0] += r[i] * r[i];
      row_reduce<WPR, 1>(ss, slots, wave, phase);
      const float rs = rstd_of(ss[0], cols, a.eps);
#pragma unroll
      for (int i = 0; i < N; ++i) r[i] = r[i] * rs * w[i];
      if (q_out) {
        // per-token INT8 codes of the unrounded n, by the rule of act_quant_int8
        // (a row with a NaN or an infinity, which no code holds, gets codes 0 and a NaN scale)
        float mx[1] = {0.f};
#pragma unroll
        for (int i = 0; i < N; ++i) mx[0] = fmaxf(mx[0], r[i] != r[i] ? __builtin_inff() : fabsf(r[i]));
        row_reduce<WPR, 1, true>(mx, slots, wave, phase);
        const bool finite = mx[0] < __builtin_inff();
        const float s = mx[0] / 127.0f;
        float q[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
          q[i] = finite && s > 0.f ? fminf(fmaxf(rintf(r[i] / s), -128.f), 127.f) : 0.f;
        R::store_codes(q_out, row, cols, tid, q);
        if (tid == 0) s_out[row] = finite ? s : __builtin_nanf("");
      } else {
        R::store(n_out, row, cols, tid, r);
      }
    }
  }
}

// Every workgroup walks rows base, base + step, ... and adds their contributions to the
// weight (and channel gate) gradients in registers; partial [groups][3][cols] holds one
// set per row group, which k_norm_grad_sum adds in order.
template <typename T, int WPR, int NV, bool VEC>
__global__ void __launch_bounds__(threads_per_wg<WPR>())
    k_block_norm_bwd(BlockNormArgs a, const void* dr, const void* dn, void* dres, void* dy, void* dgate,
                     float* partial) {
  typedef Row<T, 64 * WPR, NV, VEC> R;
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
  for (int64_t base = int64_t(blockIdx.x) * rows_per_wg<WPR>(); base < a.rows; base += step) {
    const int64_t row = base + threadIdx.x / (64 * WPR);
    if constexpr (rows_per_wg<WPR>() > 1)
      if (row >= a.rows) break;   // one wave per row: no barrier below
    float r[N], yv[N], g[N];
    float rs_y = 1.f, gt = 1.f;
    R::load(a.res, row, cols, tid, r);
    if (a.y) {
      R::load(a.y, row, cols, tid, yv);
      if (a.w_post) {
        float ss[1] = {0.f};
#pragma unroll
        for (int i = 0; i < N; ++i) ss[0] += yv[i] * yv[i];
        row_reduce<WPR, 1>(ss, slots, wave, phase);
        rs_y = rstd_of(ss[0], cols, a.eps);
      }
      if (a.gate_kind == kGateToken) {
        gt = Elem<T>::up(static_cast<const typename R::S*>(a.gate)[row]);
      } else if (a.gate_kind != kGateNone) {
        R::load(a.gate, a.gate_kind == kGateElement ? row : 0, cols, tid, g);
      }
      float w[N];
      if (a.w_post) R::load(a.w_post, 0, cols, tid, w);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        yv[i] *= rs_y;   // yh
        const float p = a.w_post ? yv[i] * w[i] : yv[i];
        r[i] += a.alpha * ((a.gate_kind == kGateChannel || a.gate_kind == kGateElement ? g[i] : gt) * p);
      }
    }
    float d[N];
    if (dr) {
      R::load(dr, row, cols, tid, d);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) d[i] = 0.f;
    }
    if (a.w_pre) {
      float dnv[N], w[N], red[2] = {0.f, 0.f};
      R::load(dn, row, cols, tid, dnv);
      R::load(a.w_pre, 0, cols, tid, w);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        red[0] += r[i] * r[i];
        red[1] += w[i] * dnv[i] * r[i];
      }
      row_reduce<WPR, 2>(red, slots, wave, phase);
      const float rs = rstd_of(red[0], cols, a.eps);
      const float c = red[1] * rs / float(cols);   // mean(w dn rh)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float rh = r[i] * rs;
        d[i] += rs * (w[i] * dnv[i] - rh * c);
        dw_pre[i] += dnv[i] * rh;
      }
    }
    R::store(dres, row, cols, tid, d);
    if (a.y) {
      float w[N], red[2] = {0.f, 0.f};
      if (a.w_post) R::load(a.w_post, 0, cols, tid, w);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float e = a.alpha * d[i];
        const float ep = e * (a.w_post ? yv[i] * w[i] : yv[i]);
        if (a.gate_kind == kGateChannel || a.gate_kind == kGateElement) {
          d[i] = e * g[i];   // dp
          if (a.gate_kind == kGateChannel) dg_ch[i] += ep;
          else g[i] = ep;
        } else {
          d[i] = e * gt;
          red[1] += ep;
        }
        if (a.w_post) {
          red[0] += d[i] * w[i] * yv[i];
          dw_post[i] += d[i] * yv[i];
        }
      }
      if (a.gate_kind == kGateElement) R::store(dgate, row, cols, tid, g);
      if (a.w_post || a.gate_kind == kGateToken) row_reduce<WPR, 2>(red, slots, wave, phase);
      if (a.gate_kind == kGateToken && tid == 0) static_cast<float*>(dgate)[row] = red[1];
      if (a.w_post) {
        const float c = red[0] / float(cols);
#pragma unroll
        for (int i = 0; i < N; ++i) d[i] = rs_y * (d[i] * w[i] - yv[i] * c);
      }
      R::store(dy, row, cols, tid, d);
    }
  }
  const int64_t group = int64_t(blockIdx.x) * rows_per_wg<WPR>() + threadIdx.x / (64 * WPR);
  float* out = partial + group * kGradSlots * cols;
  if (a.w_pre) R::store_f32(out, cols, tid, dw_pre);
  if (a.w_post) R::store_f32(out + cols, cols, tid, dw_post);
  if (a.gate_kind == kGateChannel) R::store_f32(out + 2 * cols, cols, tid, dg_ch);
}

// out[slot][c] = sum over the row groups of partial[group][slot][c]: a workgroup owns 64
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

// Workgroups of the backward pass: each keeps its sums over several rows, so that the
// partial sums (3 rows of fp32 per row group) stay small beside the rows themselves.
int bwd_groups(int64_t rows, int rpw) {
  const int64_t wgs = std::min<int64_t>((rows + rpw - 1) / rpw, 512);
  return int(wgs);
}

// Rows of up to 512 columns take one wave with one vector of 8 per lane; wider rows two
// vectors per lane and as many waves as that takes.
int waves_per_row(int64_t cols) { return cols <= 1024 ? 1 : cols <= 4096 ? 4 : cols <= 8192 ? 8 : 16; }

template <typename T, bool VEC, typename F>
hipError_t with_shape(int64_t cols, F&& f) {
  if (cols <= 512) return f(std::integral_constant<int, 1>{}, std::integral_constant<int, 1>{});
  if (cols <= 1024) return f(std::integral_constant<int, 1>{}, std::integral_constant<int, 2>{});
  if (cols <= 2048) return f(std::integral_constant<int, 4>{}, std::integral_constant<int, 1>{});
  if (cols <= 4096) return f(std::integral_constant<int, 4>{}, std::integral_constant<int, 2>{});
  if (cols <= 8192) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 2>{});
  return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 2>{});
}

template <typename F>
hipError_t with_type(int dtype, int64_t cols, F&& f) {
  const bool vec = cols % 8 == 0;
  auto go = [&](auto t, auto v) {
    typedef decltype(t) T;
    constexpr bool VEC = decltype(v)::value;
    return with_shape<T, VEC>(cols, [&](auto wpr, auto nv) { return f(t, v, wpr, nv); });
  };
  if (dtype == 0) return vec ? go(NF32{}, std::true_type{}) : go(NF32{}, std::false_type{});
  if (dtype == 1) return vec ? go(NF16{}, std::true_type{}) : go(NF16{}, std::false_type{});
  return vec ? go(NBF16{}, std::true_type{}) : go(NBF16{}, std::false_type{});
}

}  // namespace

int block_norm_max_cols() { return kMaxCols; }

hipError_t launch_block_norm(const BlockNormArgs& a, int dtype, void* r_out, void* n_out, int8_t* q_out, float* s_out,
                             hipStream_t st) {
  return with_type(dtype, a.cols, [&](auto t, auto v, auto wpr, auto nv) {
    typedef decltype(t) T;
    constexpr int WPR = decltype(wpr)::value;
    constexpr int RPW = rows_per_wg<WPR>();
    const unsigned grid = unsigned(std::min<int64_t>((a.rows + RPW - 1) / RPW, int64_t(1) << 20));
    hipLaunchKernelGGL((k_block_norm_fwd<T, WPR, decltype(nv)::value, decltype(v)::value>), dim3(grid),
                       dim3(threads_per_wg<WPR>()), 0, st, a, r_out, n_out, q_out, s_out);
    return hipGetLastError();
  });
}

int64_t block_norm_bwd_workspace(int64_t rows, int64_t cols) {
  const int wpr = waves_per_row(cols);
  const int rpw = wpr >= 4 ? 1 : 4 / wpr;
  return int64_t(bwd_groups(rows, rpw)) * rpw * kGradSlots * cols * 4;
}

hipError_t launch_block_norm_bwd(const BlockNormArgs& a, int dtype, const void* dr, const void* dn, void* dres,
                                 void* dy, float* dw_post, void* dgate, float* dw_pre, float* partial,
                                 hipStream_t st) {
  int groups = 0;
  if (a.rows > 0) {
    const hipError_t e = with_type(dtype, a.cols, [&](auto t, auto v, auto wpr, auto nv) {
      typedef decltype(t) T;
      constexpr int WPR = decltype(wpr)::value;
      const int wgs = bwd_groups(a.rows, rows_per_wg<WPR>());
      groups = wgs * rows_per_wg<WPR>();
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
