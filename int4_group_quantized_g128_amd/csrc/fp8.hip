// e4m3 products with a scale per block of 128, dense and by expert, with their quantisers.
//
//   y[t][n]  = sum_g s[g][t] ws[n / 128][g] sum_{k in g} q[t][k] wq[n][k]          g: 128 columns k
//   dx[t][k] = sum_g s[g][t] ws[g][k / 128] sum_{n in g} d[t][n] wq[n][k]          g: 128 rows n of W
//   dw[n][k] = sum_g c[g][n] x[g][k] sum_{t in g} dq[t][n] xq[t][k]                g: 128 tokens
//
// with d, dq the codes of dy along its rows and along the tokens.  One 16x16x128 matrix
// instruction takes a whole group, so each of its results is scaled once on its way into the fp32
// sums.  Within an instruction the matrix core aligns 8 products at a time to the largest and
// drops what lies 2^-13 below it, then adds in fp32: with normally distributed codes the sums are
// 1.4e-5 (relative, 2-norm) from the exact ones, which a result in 16 bits (2e-4 and up) hides and
// one in fp32 would show; results are 16 bits wide.  At worst an eight is off by 7 2^-13 of its largest
// product, a 73rd of the half step, 2^-4, by which either of its codes may be off its value.  The few-rows
// kernel, which takes all calls of up to 16 rows, widens the codes to bf16 and has no such window.
//
// Operands are read as they lie in memory: "KC" panels are contiguous along the summed index (x,
// dy and W in y), "MC" panels along their own (W in dx, both operands of dw), whose fragments come
// out of LDS through the transposing 8-byte reads; no transposed copy is made.
#include <algorithm>
#include <type_traits>

#include "e4m3.h"
#include "fp8.h"
#include "fp8_plan.h"
#include "internal.h"
#include "lds_copy.h"

namespace q4 {

namespace {

// (lambdas called from several places: their captured state, the kernel's arguments among it, has
// to stay in registers)
#define Q4_INLINE __attribute__((always_inline))

constexpr uint32_t kNoByte = 0x80000000u;   // a byte offset past every descriptor's range
typedef int32_t i32x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

struct Frag {   // 32 codes of a lane: row (column) lane % 16, k in 16 q .. + 15 and 64 + 16 q .. + 15, q = lane / 16
  u32x4_t lo, hi;
};
Q4_DEVICE f32x4_t group_product(const Frag& a, const Frag& b) {
  struct Two {
    u32x4_t lo, hi;
  };
  const i32x8_t x = bitcast<i32x8_t>(Two{a.lo, a.hi}), y = bitcast<i32x8_t>(Two{b.lo, b.hi});
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, f32x4_t{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
}

// The same through the 16-bit instructions: codes are bf16 values, and products and sums keep what
// fp32 holds of them (of 1 x 2048 x 2048 results in bf16 none is not the exact one rounded, 1.1 % with
// the instruction above).  Free where reading bounds the product, in the few-rows kernel: one row, 2048 /
// 16384, 7.3 -> 7.5 us, 2048 / 2048 4.7 -> 4.5, 16 rows 9.8 -> 9.9, 4.6 -> 4.4, 24 rows of 7168 / 4096 13.3 ->
// 13.9, 64 of 2048 / 2048 8.1 -> 8.1.  The tiles would pay for it: of 64, 1.16 times as long on average and up to
// 1.43 (64 tokens through 32 of 256 experts, whole block, 158 -> 179 us, 1280 rows of 32 experts, 7168 / 4096,
// 191 -> 232), large ones nearly twice (4096 x 7168 x 4096 with its codes 125 -> 225, forward and backward
// 4096 x 2048 x 16384 536 -> 1019, 4096 tokens through 32 of 256 experts 542 -> 906).
struct Wide {
  bf16x8_t v[4];
};
Q4_DEVICE bf16x8_t widen8(uint32_t a, uint32_t b) {
  struct Four {
    bf16x2_t v[4];
  };
  return bitcast<bf16x8_t>(Four{{__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, false),
                                 __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, true),
                                 __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, false),
                                 __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, true)}});
}
Q4_DEVICE Wide widen(const Frag& f) {
  return Wide{{widen8(f.lo[0], f.lo[1]), widen8(f.lo[2], f.lo[3]), widen8(f.hi[0], f.hi[1]), widen8(f.hi[2], f.hi[3])}};
}
Q4_DEVICE f32x4_t wide_product(const Frag& a, const Frag& b) {
  const Wide x = widen(a), y = widen(b);
  f32x4_t c = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x.v[i], y.v[i], c, 0, 0, 0);
  return c;
}

// A value that is the same in every lane, through the scalar cache (which does not count as one
// of the vector loads that the copies' waits count).
Q4_DEVICE float load_uniform(const float* p, int64_t i) {
  typedef __attribute__((address_space(4))) const float* sptr;
  return *(sptr)(uintptr_t)(p + i);
}

// Values that every lane has alike, kept in scalar registers.
Q4_DEVICE int32_t scalar(int32_t v) { return __builtin_amdgcn_readfirstlane(v); }
Q4_DEVICE uint32_t scalar(uint32_t v) { return uint32_t(__builtin_amdgcn_readfirstlane(int32_t(v))); }
Q4_DEVICE uint64_t scalar(uint64_t v) {
  return uint64_t(scalar(uint32_t(v >> 32))) << 32 | scalar(uint32_t(v));
}
Q4_DEVICE int64_t scalar(int64_t v) { return int64_t(scalar(uint64_t(v))); }

// ---------------------------------------------------------------- rows by expert
// Rows of expert x: [first, first + count), kept inside [0, t) whatever the offsets hold.
Q4_DEVICE void expert_rows(const int32_t* offsets, int x, int64_t t, int64_t& first, int64_t& count) {
  const int64_t a = offsets[x], b = offsets[x + 1];
  first = a < 0 ? 0 : a > t ? t : a;
  const int64_t end = b < 0 ? 0 : b > t ? t : b;
  count = end > first ? end - first : 0;
}

struct Span {
  int e, tile;     // expert, the tile's number over all experts
  int64_t row;     // its first row
  int rows;
};

// Row tiles of BM rows, in expert order, over a workgroup of NT threads; each thread owns a run
// of experts.
template <int NT, int BM>
struct ExpertTiles {
  int beg, end, before, own;   // this thread's experts, tiles before them, tiles of them
  int total;
  Q4_DEVICE void count(const int32_t* offsets, int e, int64_t t, int32_t* tot /* LDS [NT / 64] */) {
    const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
    const int per = (e + NT - 1) / NT;
    beg = min(e, tid * per), end = min(e, beg + per);
    own = 0;
    for (int x = beg; x < end; ++x) {
      int64_t f, c;
      expert_rows(offsets, x, t, f, c);
      own += int((c + BM - 1) / BM);
    }
    int inc = own;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(inc, o, 64);
      if (lane >= o) inc += u;
    }
    if (lane == 63) tot[wid] = inc;
    __syncthreads();
    before = inc - own, total = 0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
      if (w < wid) before += tot[w];
      total += tot[w];
    }
    __syncthreads();
  }
  // Tile `at` (below total) into *out (LDS); all threads call.
  Q4_DEVICE void find(const int32_t* offsets, int64_t t, int at, Span* out) const {
    if (at >= before && at < before + own) {
      int n = before;
      for (int x = beg; x < end; ++x) {
        int64_t f, c;
        expert_rows(offsets, x, t, f, c);
        const int nt = int((c + BM - 1) / BM);
        if (at < n + nt) {
          const int64_t r = int64_t(at - n) * BM;
          *out = Span{x, at, f + r, int(c - r < BM ? c - r : BM)};
          break;
        }
        n += nt;
      }
    }
    __syncthreads();
  }
};

// ---------------------------------------------------------------- quantisers
// A workgroup takes 16 RPT rows x 128 columns: thread i columns 8 (i % 16) .. + 7 of rows i / 16 + 16 j.
// Codes along the rows alone are bound by their bytes (4096 x 7168 bf16 17.1 us, 5.2 TB/s); with those along the
// tokens by vector instructions, 31 a value (maxima, quotients, conversions, twice) that take 86 % of the cycles
// at 4096 x 16384 (73 to 80 us, 3.4 to 3.7 TB/s) and 71 % at 8192 x 2048 (29 us).
enum Form { FORM_ROWS = 1, FORM_COLS = 2 };
// RPT of codes along the rows alone: 4096 x 7168 17.0 us (8: 22.5, 4: 19.2, 1: 16.6), 4096 x 16384
// 50.8 (52.6, 55.1, 58.7), 333 x 1040 4.0 (7.4, 4.5, 4.8); groups of tokens take 8, all 128 rows.
constexpr int kRowsAlone = 2;

template <int DT, bool GATED, int RPT>
Q4_DEVICE void load_tile(const void* x, int64_t ld, int64_t row0, int rows, int64_t c, int64_t k, float (&v)[RPT][8]) {
  typedef Elem<DT> E;
  typename E::Raw g[RPT][8 / E::VEC], u[GATED ? RPT : 1][8 / E::VEC];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int r = (threadIdx.x >> 4) + 16 * i;
    if (r < rows && c < k) {
#pragma unroll
      for (int j = 0; j < 8 / E::VEC; ++j) {
        g[i][j] = E::load(x, (row0 + r) * ld + c + j * E::VEC);
        if constexpr (GATED) u[i][j] = E::load(x, (row0 + r) * ld + k + c + j * E::VEC);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int r = (threadIdx.x >> 4) + 16 * i;
    const bool in = r < rows && c < k;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (GATED)
        v[i][j] = in ? swiglu(E::value(g[i][j / E::VEC], j % E::VEC), E::value(u[i][j / E::VEC], j % E::VEC)) : 0.f;
      else v[i][j] = in ? E::value(g[i][j / E::VEC], j % E::VEC) : 0.f;
    }
  }
}

template <int DT, int FORM, bool GATED>
__global__ void __launch_bounds__(256) k_quantize_fp8(Fp8QuantArgs a) {
  constexpr int RPT = FORM & FORM_COLS ? 8 : kRowsAlone, TILE = 16 * RPT;
  __shared__ float part[4][128];
  __shared__ Span span;
  __shared__ int32_t tot[4];
  int tile = blockIdx.x;
  int64_t row0 = int64_t(tile) * TILE, left;
  if (FORM & FORM_COLS && a.offsets) {
    ExpertTiles<256, 128> tiles;
    tiles.count(a.offsets, a.e, a.t, tot);
    if (tile >= tiles.total) return;
    tiles.find(a.offsets, a.t, tile, &span);
    row0 = span.row, left = span.rows;
  } else {
    int64_t end = a.t;
    if (a.offsets) end = std::min<int64_t>(end, std::max<int64_t>(a.offsets[a.e], 0));
    left = end - row0;
  }
  if (left <= 0) return;
  const int rows = int(std::min<int64_t>(left, TILE));
  const int cb = blockIdx.y, lane16 = threadIdx.x & 15, slot = threadIdx.x >> 4;
  const int64_t c = int64_t(cb) * 128 + lane16 * 8;
  float v[RPT][8];
  load_tile<DT, GATED, RPT>(a.x, GATED ? 2 * a.k : a.k, row0, rows, c, a.k, v);
  if constexpr (FORM & FORM_ROWS) {
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int r = slot + 16 * i;   // (the same for all lanes of a group)
      if (r < rows) {
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, magnitude(v[i][j]));
        const float s = e4m3_scale(row16_max(m));
        if (c < a.k)
          *reinterpret_cast<u32x2_t*>(a.q_row + (row0 + r) * a.k + c) = e4m3_codes8(v[i], s);
        if (lane16 == 0) a.s_row[cb * a.t + row0 + r] = s;
      }
    }
  }
  if constexpr (FORM & FORM_COLS) {
    float m[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m[j] = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) m[j] = fmaxf(m[j], magnitude(v[i][j]));
      m[j] = fmaxf(m[j], __shfl_xor(m[j], 16, 64));
      m[j] = fmaxf(m[j], __shfl_xor(m[j], 32, 64));
    }
    if ((threadIdx.x & 48) == 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) part[threadIdx.x >> 6][lane16 * 8 + j] = m[j];
    }
    __syncthreads();
    float s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int at = lane16 * 8 + j;
      s[j] = e4m3_scale(fmaxf(fmaxf(part[0][at], part[1][at]), fmaxf(part[2][at], part[3][at])));
    }
    if (c < a.k) {
      if (slot == 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) a.s_col[int64_t(tile) * a.k + c + j] = s[j];
      }
      float inv[8];
      bool plain = true;
#pragma unroll
      for (int j = 0; j < 8; ++j) inv[j] = 1.f / s[j], plain = plain && s[j] >= kPlainScale;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = slot + 16 * i;
        float q[8];
        if (plain) {
#pragma unroll
          for (int j = 0; j < 8; ++j) q[j] = e4m3_clamp(quotient(v[i][j], s[j], inv[j]));
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) q[j] = s[j] > 0.f ? e4m3_clamp(v[i][j] / s[j]) : 0.f;
        }
        if (r < rows)
          *reinterpret_cast<u32x2_t*>(a.q_col + (row0 + r) * a.k + c) =
              u32x2_t{e4m3_pack4(q[0], q[1], q[2], q[3]), e4m3_pack4(q[4], q[5], q[6], q[7])};
      }
    }
  }
}

// Bound by its bytes: 16384 x 2048 bf16 28 us, 32 matrices of 4096 x 7168 560 (5.0 TB/s), fp32 36 and 968; one
// of 2048 x 2048 7.2.
template <int DT>
__global__ void __launch_bounds__(256) k_quantize_fp8_blocks(const void* __restrict__ w, int64_t n, int64_t k,
                                                             uint32_t row_blocks, uint8_t* __restrict__ q,
                                                             float* __restrict__ s) {
  __shared__ float part[4];
  const int64_t x = blockIdx.x / row_blocks, rb = blockIdx.x - x * row_blocks;
  const int rows = int(std::min<int64_t>(128, n - rb * 128));
  const int64_t row0 = x * n + rb * 128, c = int64_t(blockIdx.y) * 128 + (threadIdx.x & 15) * 8;
  float v[8][8];
  load_tile<DT, false, 8>(w, k, row0, rows, c, k, v);
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, magnitude(v[i][j]));
  m = wave_max(m);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
  __syncthreads();
  const float sc = e4m3_scale(fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3])));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = (threadIdx.x >> 4) + 16 * i;
    if (r < rows && c < k)
      *reinterpret_cast<u32x2_t*>(q + (row0 + r) * k + c) = e4m3_codes8(v[i], sc);
  }
  if (threadIdx.x == 0) s[blockIdx.x * int64_t(gridDim.y) + blockIdx.y] = sc;
}

// ---------------------------------------------------------------- products
struct Fp8Args {
  const uint8_t *a, *b;       // token side (dw: dy) and the other operand
  int64_t lda, ldb;
  const float *sa, *sb;       // sa [groups][sa_ld]; sb: W's blocks [N / 128][K / 128] (dw: [groups][ldb])
  int64_t sa_ld, sb_ld;       // floats per row of sa and sb
  int64_t M, N, K;            // (dw: K tokens)
  int64_t b_stride, sb_stride;   // from one expert's matrix to the next
  const int32_t* offsets;     // rows by expert, or NULL
  int32_t e;
  int32_t dtype;              // of c: 1 fp16, 2 bf16
  void* c;
  int64_t ldc;
  int32_t ksplit;
  float* part;                // ksplit > 1: [ksplit][M][N]; by expert: a tile per workgroup
  int32_t tail;               // by expert, large tiles: the last tiles' K steps may be split
};

Q4_DEVICE uint16_t to16(float v, int dtype) {
  return dtype == 1 ? bitcast<uint16_t>(_Float16(v)) : bitcast<uint16_t>(__bf16(v));
}

// N values of a row (its address is a multiple of 2 alone), `count` of them inside the matrix.
template <int N>
Q4_DEVICE void store_row(void* c, int dtype, int64_t at, const float* v, int count) {
  struct __attribute__((packed, aligned(2))) Out {
    uint32_t w[N / 2];
  };
  uint16_t* p = static_cast<uint16_t*>(c) + at;
  Out o;
#pragma unroll
  for (int i = 0; i < N / 2; ++i) o.w[i] = to16(v[2 * i], dtype) | uint32_t(to16(v[2 * i + 1], dtype)) << 16;
  if (count >= N) {
    *reinterpret_cast<Out*>(p) = o;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < count) p[i] = uint16_t(o.w[i / 2] >> (16 * (i % 2)));
  }
}

// R rows (MC: columns) of one operand, one K step of 128 codes: 128 R bytes in copies of 1 KB.
// 16-byte chunks are XOR-swizzled so that fragment reads hit distinct banks:
//   KC  [R][128]: chunk c of row r at c ^ ((r / 2) % 8)
//   MC  [128][R]: chunk c of row k at c ^ f(k), f from the bits of k in which the 16 rows that two
//       quarters of a transposing read touch differ.
template <bool MC, int R>
struct Panel8 {
  static constexpr int BYTES = R * 128;
  static constexpr int COPIES = BYTES / 1024;
  static constexpr int CPR = MC ? R / 16 : 8;

  static Q4_DEVICE int swz(int r) {
    if constexpr (!MC) return (r >> 1) & 7;
    else if constexpr (R == 256) return (r & 7) | ((r >> 4) & 1) << 3;
    else if constexpr (R == 128) return ((r >> 1) & 3) | ((r >> 4) & 1) << 2;
    else return ((r >> 2) & 1) | ((r >> 4) & 1) << 1;
  }
  // Rows (MC: of k) per copy; which of two swizzles copy j (of a wave's, the first a multiple of
  // their number) has, and the first copy that has it.
  static constexpr int ROWS = 64 / CPR;
  static constexpr int odd(int j) { return MC && R == 128 ? (j >> 1) & 1 : j & 1; }
  static constexpr int copy_of(int odd) { return MC && R == 128 ? 2 * odd : odd; }
  // Byte offset of the lane's chunk of copy `copy` from the panel's first row and first k of the
  // step.  `left`: KC, codes of K left at the step; MC, columns left at the first column.
  static Q4_DEVICE uint32_t offset(int copy, int lane, int64_t ld, int64_t left) {
    const int id = copy * 64 + lane, r = id / CPR, c = (id % CPR) ^ swz(r);
    return c * 16 < left ? uint32_t(r * ld + c * 16) : kNoByte;
  }
  struct Feed {   // what is left of the panel from the next K step on
    uint64_t addr;
    int64_t left;
    uint32_t inc;
    Q4_DEVICE u32x4_t rsrc(bool valid) const {
      const uint32_t n = !valid || left <= 0 ? 0u : left > 0x7fffffff ? 0x7fffffffu : uint32_t(left);
      return u32x4_t{uint32_t(addr), uint32_t(addr >> 32) & 0xffffu, n, 0x00020000u};
    }
    Q4_DEVICE void next() { addr += inc, left -= inc; }
  };
  // The panel from row (MC: column) row0 on of `rows` rows x K codes, at step `step`.
  static Q4_DEVICE Feed feed(const uint8_t* p, int64_t ld, int64_t rows, int64_t K, int64_t row0, int step) {
    const uint32_t inc = MC ? uint32_t(ld) * 128u : 128u;
    const int64_t at = (MC ? row0 : row0 * ld) + int64_t(step) * inc;
    return Feed{reinterpret_cast<uint64_t>(p) + at, (MC ? K * ld : rows * ld) - at, inc};
  }

  static Q4_DEVICE uint32_t lane_base(int lane) {
    const int q = lane >> 4, s = lane & 15;
    if constexpr (!MC) return s * 128 + ((q ^ swz(s)) << 4);
    else return (16 * q + (s >> 1)) * R + (swz(16 * q + (s >> 1)) << 4) + ((s & 1) << 3);
  }
  // The same through addresses kept in registers, with constant offsets: `at` panel bytes on, rows
  // (columns) r0 (a constant, MC: below 64) on.  MC: the panel's LDS address is a multiple of 64.
  struct Reader {
    uint32_t lo, hi;
    Q4_DEVICE void start(uint32_t lds, int lane, int first) {   // first: a multiple of 16 (MC: of 64)
      const uint32_t lb = lane_base(lane);
      lo = MC ? lds + (lb ^ first) : lds + first * 128 + lb;
      hi = lds + first * 128 + (lb ^ 64);
    }
    Q4_DEVICE void move(int32_t by) { lo += by, hi += by; }
    Q4_DEVICE Frag read(int at, int r0) const {
      Frag f;
      if constexpr (!MC) {
        typedef __attribute__((address_space(3))) const u32x4_t* lptr;
        f.lo = *((lptr)(uintptr_t)lo + (at + r0 * 128) / 16);
        f.hi = *((lptr)(uintptr_t)hi + (at + r0 * 128) / 16);
      } else {
        return frag(at, lo, r0);
      }
      return f;
    }
  };
  // Fragment of rows (columns) r0 .. r0 + 15 of the panel at LDS address `lds`.
  static Q4_DEVICE Frag frag(uint32_t lds, uint32_t lb, int r0) {
    Frag f;
    if constexpr (!MC) {
      typedef __attribute__((address_space(3))) const u32x4_t* lptr;
      f.lo = *(lptr)(uintptr_t)(lds + r0 * 128 + lb);
      f.hi = *(lptr)(uintptr_t)(lds + r0 * 128 + (lb ^ 64));
    } else {
      // a 16-lane group reads 8 rows k x 16 columns and each lane gets its column's 8 codes
      typedef int32_t i32x2 __attribute__((ext_vector_type(2)));
      typedef __attribute__((address_space(3))) i32x2* lptr;
      const uint32_t at = lds + (lb ^ r0);
      u32x2_t v[4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
        v[r] = bitcast<u32x2_t>(
            __builtin_amdgcn_ds_read_tr8_b64_v2i32((lptr)(uintptr_t)(at + (8 * (r & 1) + 64 * (r >> 1)) * R)));
      f.lo = u32x4_t{v[0][0], v[0][1], v[1][0], v[1][1]};
      f.hi = u32x4_t{v[2][0], v[2][1], v[3][0], v[3][1]};
    }
    return f;
  }
};

template <typename P, int N>
Q4_DEVICE void copies8(const u32x4_t& rs, uint32_t at, int first, int lane, int64_t ld, int64_t left) {
  static_assert(N % 2 == 0, "two copies at a time");
#pragma unroll
  for (int j = 0; j < N; j += 2)
    copy2_to_lds(rs, at + (first + j) * 1024, P::offset(first + j, lane, ld, left),
                 P::offset(first + j + 1, lane, ld, left));
}

template <int N>
Q4_DEVICE void wait_barrier8() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// Scales of one step, 4 bytes per row, beside the panels.
struct ScaleFeed {
  uint64_t addr;
  int64_t inc;
  uint32_t bytes;
  Q4_DEVICE u32x4_t rsrc(bool valid) const {
    return u32x4_t{uint32_t(addr), uint32_t(addr >> 32) & 0xffffu, valid ? bytes : 0u, 0x00020000u};
  }
  Q4_DEVICE void next() { addr += inc; }
  static Q4_DEVICE ScaleFeed of(const float* s, int64_t ld, int64_t group, int64_t row0, int64_t rows) {
    return ScaleFeed{reinterpret_cast<uint64_t>(s + group * ld + row0), ld * 4,
                     rows <= 0 ? 0u : uint32_t(rows > 256 ? 1024 : rows * 4)};
  }
};

// What a workgroup multiplies: rows m0 .. m_end - 1 (at most BM of them) by columns from n0 on, K
// steps s_begin .. s_end - 1 of expert x (0: the only matrix).
struct Work {
  int64_t m0, m_end, n0;
  int64_t k_first, k_rows;   // the summed index's range (dw by expert: the expert's tokens)
  int64_t group0;            // its first group (dw)
  int x, slice, s_begin, s_end;
  int32_t part;              // >= 0: some K steps of a tile, whose sums go there to be joined later
};

// By expert, the grid's workgroups walk the tiles that the offsets make; else each has one.
// Workgroup b runs on XCD b % 8.  Tiles are numbered in bands of 8 row tiles that walk the column
// tiles together, and a round of an XCD's workgroups is a run of them (its L2 keeps the panels
// they share); the XCDs take the runs in turn, since experts of few rows make cheap ones.
//
// How many tiles there are follows from the offsets, which the host does not know, and a last
// round of few tiles takes as long as a full one.  So where the tiles that an XCD has left are at
// most half as many as its workgroups, they are split along K, as many slices as workgroups
// allow; each workgroup stores the sums of its one slice, and k_fp8_tail adds them (32 experts of 128
// rows and one of 300, 7168 / 4096: 298 -> 257 us).
template <int MODE, int NT, int BM, int BN>
struct Tiles {
  ExpertTiles<NT, MODE == FP8_DW ? 128 : BM> experts;
  uint32_t mtiles, ntiles, plane;
  uint32_t wgs;                   // workgroups of an XCD
  uint32_t full, slices, limit;   // items from `full` on, below `limit`, are `slices` each of a tile
  uint32_t start;                 // tile of the first of them
  Span* span;

  Q4_DEVICE Tiles(const Fp8Args& g, uint32_t mt, uint32_t nt, uint32_t per_xcd, Span* sp, int32_t* tot)
      : ntiles(nt), wgs(per_xcd), span(sp) {
    if (g.offsets) experts.count(g.offsets, g.e, MODE == FP8_DW ? g.K : g.M, tot);
    mtiles = MODE != FP8_DW && g.offsets ? uint32_t(experts.total) : mt;
    plane = mtiles * ntiles;
    const uint32_t total = plane * (MODE == FP8_DW ? uint32_t(g.e) : 1u) * uint32_t(g.ksplit);
    const uint32_t xcd = blockIdx.x % 8, whole = total / (8 * wgs), rest = total - whole * 8 * wgs;
    const uint32_t left = rest / 8 + (xcd < rest % 8 ? 1u : 0u);
    plane = scalar(plane), mtiles = scalar(mtiles);
    full = scalar(whole * wgs), start = scalar(whole * 8 * wgs + xcd * (rest / 8) + min(xcd, rest % 8));
    slices = 1;
    if (MODE != FP8_DW && g.tail && left)
      slices = scalar(uint32_t(max(1, fp8_tail_slices(wgs / left, int((g.K + 127) / 128)))));
    limit = scalar(full + left * slices);
  }
  // The items of a workgroup: one of each round, and no tile's place among the XCD's twice, so that
  // the workgroups that get row tiles of few rows are not the same in every round.
  Q4_DEVICE uint32_t item(uint32_t round) const { return round * wgs + (blockIdx.x / 8 + round) % wgs; }
  // All threads call; item: 0 .. limit - 1 of this XCD.
  Q4_DEVICE Work at(const Fp8Args& g, uint32_t item) const {
    const bool last = item >= full, part = MODE != FP8_DW && last && slices > 1;
    const uint32_t round = item / wgs;
    uint32_t i = last ? start + (item - full) / slices : (round * 8 + blockIdx.x % 8) * wgs + item - round * wgs;
    const uint32_t z = i / plane;   // expert (dw) or K slice
    i -= z * plane;
    constexpr uint32_t GM = 8;
    const uint32_t band = i / (GM * ntiles), b0 = band * GM, gm = mtiles - b0 < GM ? mtiles - b0 : GM;
    i -= band * GM * ntiles;
    const uint32_t mt = b0 + i % gm, nt = i / gm;
    Work w{int64_t(mt) * BM, g.M, int64_t(nt) * BN, 0, g.K, 0, 0, 0, 0, 0, part ? int32_t(scalar((item - full) * 8 + blockIdx.x % 8)) : -1};
    if (MODE != FP8_DW && g.offsets) {
      experts.find(g.offsets, g.M, int(mt), span);
      w.x = span->e;
      w.m0 = span->row;
      w.m_end = w.m0 + span->rows;
    } else if (MODE == FP8_DW && g.offsets) {
      w.x = int(z);
      expert_rows(g.offsets, w.x, g.K, w.k_first, w.k_rows);
      // the expert's first group: those of the threads before its owner and of the owner's run
      if (w.x >= experts.beg && w.x < experts.end) {
        int n = experts.before;
        for (int y = experts.beg; y < w.x; ++y) {
          int64_t f, c;
          expert_rows(g.offsets, y, g.K, f, c);
          n += int((c + 127) / 128);
        }
        span->tile = n;
      }
      __syncthreads();
      w.group0 = span->tile;
      // (offsets that are not ascending may count more groups than the scales have room for)
      const int64_t room = g.K / 128 + std::min<int64_t>(g.e, g.K) - w.group0;
      w.k_rows = std::min<int64_t>(w.k_rows, std::max<int64_t>(room, 0) * 128);
    }
    const int all = int((w.k_rows + 127) / 128), split = part ? int(slices) : g.ksplit, per = (all + split - 1) / split;
    w.slice = part ? int((item - full) % slices) : g.ksplit > 1 ? int(z) : 0;
    w.s_begin = min(all, w.slice * per), w.s_end = min(all, w.s_begin + per);
    w.m0 = scalar(w.m0), w.m_end = scalar(w.m_end), w.n0 = scalar(w.n0), w.k_first = scalar(w.k_first);
    w.k_rows = scalar(w.k_rows), w.group0 = scalar(w.group0), w.x = scalar(w.x), w.slice = scalar(w.slice);
    w.s_begin = scalar(w.s_begin), w.s_end = scalar(w.s_end);
    return w;
  }
};

// W's block scales of a wave's columns.
template <int MODE>
struct BlockScale {
  const float* s;
  int64_t step;
  Q4_DEVICE BlockScale(const Fp8Args& g, const Work& w, int64_t n) {
    const int64_t nb = std::min<int64_t>(n, g.N - 1) / 128;
    s = g.sb + w.x * g.sb_stride + (MODE == FP8_Y ? nb * g.sb_ld : nb);
    step = MODE == FP8_Y ? 1 : g.sb_ld;
  }
  Q4_DEVICE float at(int k) const {
    if constexpr (MODE == FP8_DW) return 1.f;
    else return load_uniform(s, k * step);
  }
};

// The end of a tile: sums of rows m (lane % 16 of each 16), columns n + 16 b + 4 (lane / 16) .. + 3.
// A K slice's, as they are:
template <int MB, int NB>
Q4_DEVICE void store_slice(const Fp8Args& g, const Work& w, const f32x4_t (&acc)[MB][NB], int64_t m, int64_t n, int lane) {
#pragma unroll
  for (int a = 0; a < MB; ++a) {
    const int64_t row = m + 16 * a + (lane & 15);
    if (row >= w.m_end) continue;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int64_t col = n + 16 * b + 4 * (lane >> 4);
      float* o = g.part + (int64_t(w.slice) * g.M + row) * g.N + col;
      if (col + 4 <= g.N && (g.N & 3) == 0) {
        *reinterpret_cast<f32x4_t*>(o) = acc[a][b];
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (col + e < g.N) o[e] = acc[a][b][e];
      }
    }
  }
}

// The result, through `turn`, the wave's part of LDS:
template <int MODE, int MB, int NB>
Q4_DEVICE void finish(const Fp8Args& g, const Work& w, const f32x4_t (&acc)[MB][NB], int64_t m, int64_t n, uint32_t turn,
                      int lane) {
  constexpr int COLS = 16 * NB;
  if (g.ksplit > 1) return store_slice<MB, NB>(g, w, acc, m, n, lane);
  // through the wave's part of LDS, 32 rows at a time, so that a lane stores 8 columns of one row;
  // 16-byte chunk c of row r lies at c ^ (r % chunks of a row)
  constexpr int CH = COLS / 4, LPR = COLS / 8;
  typedef __attribute__((address_space(3))) f32x4_t* lptr;
  void* c = g.c;
  if (MODE == FP8_DW) c = static_cast<uint16_t*>(c) + w.x * g.M * g.ldc;
#pragma unroll
  for (int h = 0; h < MB / 2; ++h) {
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int r = 16 * a + (lane & 15), ch = 4 * b + (lane >> 4);
        *(lptr)(uintptr_t)(turn + r * (COLS * 4) + ((ch ^ (r & (CH - 1))) << 4)) = acc[2 * h + a][b];
      }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int r0 = 0; r0 < 32; r0 += 64 / LPR) {
      const int r = r0 + lane / LPR, ch = 2 * (lane % LPR);
      const f32x4_t u = *(lptr)(uintptr_t)(turn + r * (COLS * 4) + ((ch ^ (r & (CH - 1))) << 4));
      const f32x4_t v = *(lptr)(uintptr_t)(turn + r * (COLS * 4) + (((ch + 1) ^ (r & (CH - 1))) << 4));
      const int64_t row = m + 32 * h + r, col = n + 4 * ch;
      const float o[8] = {u[0], u[1], u[2], u[3], v[0], v[1], v[2], v[3]};
      if (row < w.m_end && col < g.N)
        store_row<8>(c, g.dtype, row * g.ldc + col, o, int(std::min<int64_t>(8, g.N - col)));
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}

// Two values of a row as 16 bits.
template <bool F16>
Q4_DEVICE uint32_t pack2(float a, float b) {
  if constexpr (F16) return bitcast<uint16_t>(_Float16(a)) | uint32_t(bitcast<uint16_t>(_Float16(b))) << 16;
  else return bitcast<uint16_t>(__bf16(a)) | uint32_t(bitcast<uint16_t>(__bf16(b))) << 16;
}

// The same for 64 columns without LDS: 4 x 4 transposes over the lanes' quarters and the four
// blocks (swaps of half waves, then of quarters) leave a lane 16 columns of its row, 32 bytes,
// four lanes a whole line.
template <int MODE, int MB, bool F16>
Q4_DEVICE void finish64(const Fp8Args& g, const Work& w, const f32x4_t (&acc)[MB][4], int64_t m, int64_t n, int lane) {
  struct __attribute__((packed, aligned(2))) Out {
    uint32_t w[4];
  };
  const int64_t col = n + 16 * (lane >> 4);
  const int rows = int(std::min<int64_t>(w.m_end - m, 16 * MB)) - (lane & 15);   // below: 16 a
  const int cols = int(std::min<int64_t>(g.N - col, 16));
  uint16_t* c = static_cast<uint16_t*>(g.c) + (MODE == FP8_DW ? w.x * g.M * g.ldc : 0) + (m + (lane & 15)) * g.ldc + col;
  const int64_t down = 16 * g.ldc;
#pragma unroll
  for (int a = 0; a < MB; ++a, c += down) {
    uint32_t o[8];   // piece p (columns 4 p .. + 3) of the lane's block: o[2 p], o[2 p + 1]
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      uint32_t v[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) v[b] = pack2<F16>(acc[a][b][2 * d], acc[a][b][2 * d + 1]);
      const auto x = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
      const auto y = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
      const auto p01 = __builtin_amdgcn_permlane16_swap(x[0], y[0], false, false);
      const auto p23 = __builtin_amdgcn_permlane16_swap(x[1], y[1], false, false);
      o[d] = p01[0], o[2 + d] = p01[1], o[4 + d] = p23[0], o[6 + d] = p23[1];
    }
    if (16 * a >= rows) continue;
    if (cols == 16) {
      *reinterpret_cast<Out*>(c) = Out{{o[0], o[1], o[2], o[3]}};
      *reinterpret_cast<Out*>(c + 8) = Out{{o[4], o[5], o[6], o[7]}};
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (e < cols) c[e] = uint16_t(o[e / 2] >> (16 * (e % 2)));
    }
  }
}

// BM x BN per workgroup of WM x WN waves, a ring of NS K steps in LDS: step s + NS - 1 is copied
// while step s is multiplied, one barrier per step.  Three steps of 64 x 64 let a CU hold three
// workgroups; a lone one takes 0.4 us a step, the 16 KB that its CU reads (rings of 5 and 8 steps,
// and two steps per barrier, were no faster).  64 x 7168 x 4096 in 4 K slices 11.6 us: 14 steps, 5.6 us, and the
// start and end of 256 lone workgroups, with 4 MB of slices stored.
template <int MODE, int BM, int BN, int WM, int WN, int NS>
__global__ void __launch_bounds__(64 * WM * WN) k_fp8(Fp8Args g, uint32_t mtiles, uint32_t ntiles) {
  constexpr bool AMC = MODE == FP8_DW, BMC = MODE != FP8_Y, VECB = MODE == FP8_DW;
  constexpr int NW = WM * WN, NT = 64 * NW;
  typedef Panel8<AMC, BM> PA;
  typedef Panel8<BMC, BN> PB;
  constexpr int SCALES = (BM + (VECB ? BN : 0)) * 4;
  constexpr int STAGE = PA::BYTES + PB::BYTES + SCALES;
  constexpr int CA = PA::COPIES / NW, CB = PB::COPIES / NW, CPW = CA + CB + 1 + (VECB ? 1 : 0);
  constexpr int MB = BM / WM / 16, NB = BN / WN / 16, COLS = NB * 16;
  constexpr int AHEAD = NS - 1;
  static_assert(BN / WN <= 64, "a wave's columns lie in one block of W");
  static_assert(NS * STAGE >= NW * 32 * COLS * 4, "the turn at a tile's end");
  __shared__ __align__(16) uint8_t ring[NS * STAGE];
  __shared__ Span span;
  __shared__ int32_t tot[NW];

  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  const int wm = wid % WM, wn = wid / WM;
  const uint32_t lds0 = lds_addr(ring);
  const uint32_t lba = PA::lane_base(lane), lbb = PB::lane_base(lane);
  const Tiles<MODE, NT, BM, BN> tiles(g, mtiles, ntiles, (gridDim.x + 7) / 8, &span, tot);
  for (uint32_t round = 0; tiles.item(round) < tiles.limit; ++round) {
    const Work w = tiles.at(g, tiles.item(round));
    const uint8_t* ap = g.a + (MODE == FP8_DW ? w.k_first * g.lda : 0);
    const uint8_t* bp = g.b + (MODE == FP8_DW ? w.k_first * g.ldb : w.x * g.b_stride);
    typename PA::Feed fda = PA::feed(ap, g.lda, w.m_end, w.k_rows, w.m0, w.s_begin);
    typename PB::Feed fdb = PB::feed(bp, g.ldb, g.N, w.k_rows, w.n0, w.s_begin);
    ScaleFeed fsa = ScaleFeed::of(g.sa, g.sa_ld, w.group0 + w.s_begin, w.m0, w.m_end - w.m0);
    ScaleFeed fsb = ScaleFeed::of(g.sb, g.sb_ld, w.group0 + w.s_begin, w.n0, g.N - w.n0);
    const BlockScale<MODE> block(g, w, w.n0 + wn * COLS);
    int64_t k_left = w.k_rows - int64_t(w.s_begin) * 128;
    int si = w.s_begin, slot_in = 0;
    auto issue = [&]() {
      const bool in = si < w.s_end;
      const uint32_t at = lds0 + slot_in * STAGE;
      copies8<PA, CA>(fda.rsrc(in), at, wid * CA, lane, g.lda, AMC ? g.M - w.m0 : k_left);
      copies8<PB, CB>(fdb.rsrc(in), at + PA::BYTES, wid * CB, lane, g.ldb, BMC ? g.N - w.n0 : k_left);
      // (64 scales a copy; waves beyond the panel's repeat a copy)
      const int ca = wid % (BM / 64), cb = wid % (BN / 64);
      copy4_to_lds(fsa.rsrc(in), at + PA::BYTES + PB::BYTES + ca * 256, (ca * 64 + lane) * 4);
      if constexpr (VECB)
        copy4_to_lds(fsb.rsrc(in), at + PA::BYTES + PB::BYTES + BM * 4 + cb * 256, (cb * 64 + lane) * 4);
      fda.next(), fdb.next(), fsa.next(), fsb.next();
      k_left -= 128;
      ++si;
      slot_in = slot_in == NS - 1 ? 0 : slot_in + 1;
    };

    f32x4_t acc[MB][NB];
#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[a][b] = f32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) issue();
    float sb_next = w.s_begin < w.s_end ? block.at(w.s_begin) : 0.f;
    int slot = 0;
    for (int s = w.s_begin; s < w.s_end; ++s) {
      wait_barrier8<(AHEAD - 1) * CPW>();
      const uint32_t base = lds0 + slot * STAGE;
      slot = slot == NS - 1 ? 0 : slot + 1;
      const float sbs = sb_next;
      if (s + 1 < w.s_end) sb_next = block.at(s + 1);
      typedef __attribute__((address_space(3))) const float* fptr;
      typedef __attribute__((address_space(3))) const f32x4_t* vptr;
      const uint32_t sc = base + PA::BYTES + PB::BYTES;
      Frag fa[MB], fb[NB];
      float sa[MB];
      f32x4_t vb[VECB ? NB : 1];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        fb[b] = PB::frag(base + PA::BYTES, lbb, wn * COLS + 16 * b);
        if constexpr (VECB) vb[b] = *(vptr)(uintptr_t)(sc + (BM + wn * COLS + 16 * b + 4 * (lane >> 4)) * 4);
      }
#pragma unroll
      for (int a = 0; a < MB; ++a) {
        fa[a] = PA::frag(base, lba, wm * (BM / WM) + 16 * a);
        sa[a] = *(fptr)(uintptr_t)(sc + (wm * (BM / WM) + 16 * a + (lane & 15)) * 4);
      }
      issue();
#pragma unroll
      for (int a = 0; a < MB; ++a)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const f32x4_t p = group_product(fb[b], fa[a]);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[a][b][e] = __builtin_fmaf(p[e], sa[a] * (VECB ? vb[b][e] : sbs), acc[a][b][e]);
        }
    }
    wait_barrier8<0>();   // every wave's copies and reads are done: LDS is free
    finish<MODE, MB, NB>(g, w, acc, w.m0 + wm * (BM / WM), w.n0 + wn * COLS, lds0 + wid * (32 * COLS * 4), lane);
    __syncthreads();   // LDS is read to its end: the next tile's copies may land
  }
}

// Large tiles: BM x BN per workgroup of WM x WN waves with one barrier per K step and copies
// SLOTS - 1 whole steps ahead, so that the matrix core never waits for a step to begin.
// A's panel lies in two halves: A0 the first half of every wave's rows, A1 the second.  Wave tiles
// are walked row block by row block; each block's products run while the next block's fragment is
// read and the last block's results are scaled into the sums.  In step s
//   block MB / 2 - 1 begins with the barrier: every wave has read B and A0 of step s and A1 of
//     step s - 1, and A1 of s and B and A0 of s + 1 are in LDS; then the copies of A1 of
//     s + SLOTS - 1 and of B and A0 of s + SLOTS go into the places that are free;
//   the last block ends with the reads of B and of A0's first block of step s + 1.
// A workgroup's next tile is on its way while the results of one are stored.  (Everything that has
// one value per workgroup is kept in scalar registers and every helper inlined: as soon as the
// arguments went through memory the loops spilled, dw of 4096 x 7168 x 4096 141 -> 233 us.)
//
// 4096 x 7168 x 4096 takes 108 us (2.2 PFLOP/s), 4096 x 2048 x 16384 143 to 175 (1.6 to 1.9): y 143, dx 131
// and dW 156 on an idle card, up to 175, 158 and 190 in a row of passes, when the clock falls to 1.9 GHz.
// The matrix core is busy 54 % of the cycles there, here 46 (y), 52 (dx) and 43 (dW); the vector
// instructions take 37, 39, 34 and 50 % more.  The loops have 5.0 (y), 4.9 (dx) and 8.5 (dW) of them to a
// matrix instruction, 4, 4 and 8 of which are the scaled sums, and the two units hardly overlap: their
// sum is 85 to 94 % of the cycles, in the order of the products' times.  LDS reads take 21 to 24 %,
// without bank conflicts.
template <int MODE, int BM, int BN, int WM, int WN, int SLOTS>
__global__ void __launch_bounds__(64 * WM * WN, 512 / (64 * WM * WN)) k_fp8_big(Fp8Args g, uint32_t mtiles, uint32_t ntiles) {
  constexpr bool AMC = MODE == FP8_DW, BMC = MODE != FP8_Y, VECB = MODE == FP8_DW;
  constexpr int NW = WM * WN, NT = 64 * NW;
  constexpr int HR = BM / 2, HW = HR / WM;   // rows of half a panel, of it a wave's
  typedef Panel8<AMC, HR> PA;
  typedef Panel8<BMC, BN> PB;
  constexpr int CA = PA::COPIES / NW, CB = PB::COPIES / NW;
  constexpr int MB = BM / WM / 16, NB = BN / WN / 16, COLS = NB * 16;
  // LDS: B of every slot, A0, A1, then the scales: A0's, A1's, B's
  constexpr int A0 = SLOTS * PB::BYTES, A1 = A0 + SLOTS * PA::BYTES, S0 = A1 + SLOTS * PA::BYTES;
  constexpr int S1 = S0 + SLOTS * HR * 4, SB = S1 + SLOTS * HR * 4, BYTES = SB + (VECB ? SLOTS * BN * 4 : 0);
  static_assert(HR % 64 == 0 && CA >= 1 && CB >= 1 && MB >= 4, "");
  static_assert(COLS == 64, "a wave's columns lie in one block of W, and finish64");
  // (a Reader's transposing reads flip bits 4 and 5 of LDS addresses: every panel starts at a multiple of 64)
  __shared__ __align__(128) uint8_t mem[BYTES];
  static_assert(A0 % 64 == 0 && A1 % 64 == 0 && PA::BYTES % 64 == 0 && PB::BYTES % 64 == 0, "");
  __shared__ Span span;
  __shared__ int32_t tot[NW];

  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  const int wm = wid / WN, wn = wid % WN;   // (a SIMD's two waves in different rows)
  const uint32_t lds0 = lds_addr(mem);
  const Tiles<MODE, NT, BM, BN> tiles(g, mtiles, ntiles, (gridDim.x + 7) / 8, &span, tot);
  uint32_t round = 0, item = scalar(tiles.item(0));
  if (item >= tiles.limit) return;
  Work w = tiles.at(g, item);
  const uint32_t lda = uint32_t(g.lda), ldb = uint32_t(g.ldb);
  // what a tile's copies need
  int steps;
  int32_t k_all, a_left, b_left;
  uint32_t oa[2], oa1[2], ob[2], s_rows;   // (by swizzle; MC: oa1 of half 1)
  int chunk[2];   // KC: the chunk's first code in the step
  uint64_t a_at, b_at, sa_at, sb_at;
  auto aim = [&]() Q4_INLINE {
    // (nothing that follows from the lane alone is worth a register through the tiles' loop)
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    const uint8_t* ap = g.a + (MODE == FP8_DW ? w.k_first * g.lda : 0);
    const uint8_t* bp = g.b + (MODE == FP8_DW ? w.k_first * g.ldb : w.x * g.b_stride);
    // Row r of half h is row (r / HW) 2 HW + h HW + r % HW of the tile; the rows (MC: the lane's
    // columns) of a copy lie in one wave's part.
    steps = scalar(w.s_end - w.s_begin);
    k_all = scalar(int32_t(w.k_rows - int64_t(w.s_begin) * 128));   // (below 2^31: t, n and k are)
    a_left = scalar(int32_t(std::min<int64_t>(AMC ? g.M - w.m0 : w.m_end - w.m0, BM)));
    b_left = scalar(int32_t(std::min<int64_t>(g.N - w.n0, BN)));
    s_rows = uint32_t(scalar(int32_t(std::min<int64_t>(w.m_end - w.m0, BM)))) * 4;
    // byte offsets of a lane's chunk from the panel's start at the step (KC: without the first row)
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const int ia = wid * CA + (CA > 1 ? PA::copy_of(v) : 0), ra0 = (ia * 64 + lane) / PA::CPR;
      const int ca = (lane % PA::CPR) ^ PA::swz(ra0);
      if (AMC) {
        const uint32_t row = uint32_t(ra0 - (CA > 1 ? PA::copy_of(v) : 0) * PA::ROWS) * lda;
        const int at = ca * 16 + ca * 16 / HW * HW;
        oa[v] = at < a_left ? row + at : kNoByte;
        oa1[v] = at + HW < a_left ? row + at + HW : kNoByte;
      } else {
        oa[v] = uint32_t(lane / PA::CPR) * lda + ca * 16;
        chunk[v] = ca * 16;
      }
      const int ib = wid * CB + PB::copy_of(v), rb0 = (ib * 64 + lane) / PB::CPR;
      const int cb = (lane % PB::CPR) ^ PB::swz(rb0);
      if (BMC) ob[v] = cb * 16 < b_left ? uint32_t(rb0 - PB::copy_of(v) * PB::ROWS) * ldb + cb * 16 : kNoByte;
      else ob[v] = uint32_t(lane / PB::CPR) * ldb + cb * 16, chunk[v] = cb * 16;   // (as in A's copies)
    }
    a_at = scalar(uint64_t(reinterpret_cast<uint64_t>(ap) + (AMC ? w.m0 : w.m0 * g.lda) + w.s_begin * (AMC ? g.lda * 128 : 128)));
    b_at = scalar(uint64_t(reinterpret_cast<uint64_t>(bp) + (BMC ? w.n0 : w.n0 * g.ldb) + w.s_begin * (BMC ? g.ldb * 128 : 128)));
    sa_at = scalar(uint64_t(reinterpret_cast<uint64_t>(g.sa + (w.group0 + w.s_begin) * g.sa_ld + w.m0)));
    sb_at = scalar(uint64_t(reinterpret_cast<uint64_t>(g.sb + (VECB ? (w.group0 + w.s_begin) * g.sb_ld + w.n0 : 0))));
  };
    // The panel of step i: what the descriptor covers ends with the panel's last row (KC: of the
    // tile, MC: of the step), so that rows beyond read as zeros; past the last step it is empty.
    auto rsrc = [](uint64_t at, uint32_t bytes) {
      return u32x4_t{uint32_t(scalar(int32_t(uint32_t(at)))), uint32_t(scalar(int32_t(at >> 32))) & 0xffffu,
                     uint32_t(scalar(int32_t(bytes))), 0x00020000u};
    };
    auto range = [&](bool mc, int i, uint32_t rows, uint32_t ld) Q4_INLINE -> uint32_t {
      if (i < 0 || i >= steps) return 0;
      return mc ? uint32_t(min(128, k_all - i * 128)) * ld : rows * ld - uint32_t(w.s_begin + i) * 128;
    };
    // KC: chunks past K's end take no byte
    auto inside = [&](int i, uint32_t o, int odd) Q4_INLINE { return chunk[odd] < k_all - i * 128 ? o : kNoByte; };
    // Copy j of step i (0: s_begin) of half h of A, of B, into a slot.
    auto copy_a = [&](int i, int slot, int h, int j) Q4_INLINE {
      uint32_t o;
      if constexpr (AMC) {
        o = (h ? oa1 : oa)[PA::odd(j)] + j * PA::ROWS * lda;   // (kNoByte stays beyond every range)
      } else {
        const int r = (wid * CA + j) * PA::ROWS;
        o = inside(i, oa[PA::odd(j)], PA::odd(j)) + uint32_t(r + r / HW * HW + h * HW) * lda;
      }
      const uint64_t at = a_at + int64_t(i) * (AMC ? g.lda * 128 : 128);
      copy_to_lds(rsrc(at, range(AMC, i, a_left, lda)), lds0 + (h ? A1 : A0) + slot * PA::BYTES + (wid * CA + j) * 1024, o);
    };
    auto copy_b = [&](int i, int slot, int j) Q4_INLINE {
      uint32_t o = ob[PB::odd(j)];
      if constexpr (BMC) o += j * PB::ROWS * ldb;
      else o = inside(i, o, PB::odd(j)) + uint32_t((wid * CB + j) * PB::ROWS) * ldb;
      const uint64_t at = b_at + int64_t(i) * (BMC ? g.ldb * 128 : 128);
      copy_to_lds(rsrc(at, range(BMC, i, b_left, ldb)), lds0 + slot * PB::BYTES + (wid * CB + j) * 1024, o);
    };
    // Scales, 64 a copy and one copy a wave: of a half of A (half 1 one step before half 0, as the
    // panels), of B.  (Waves beyond their number repeat a copy.)
    const int sh = wid & 1, sc = (wid >> 1) % (HR / 64);
    const uint32_t s_off = uint32_t(sc * 64 + lane + (sc * 64 + lane) / HW * HW + sh * HW) * 4;
    auto copy_sa = [&](int i, int slot, int before) Q4_INLINE {   // half 0 of step i or half 1 of step i - 1
      const int k = i - sh;
      copy4_to_lds(rsrc(sa_at + int64_t(k) * g.sa_ld * 4, k >= 0 && k < steps ? s_rows : 0),
                   lds0 + (sh ? S1 : S0) + (sh ? before : slot) * (HR * 4) + sc * 256, s_off);
    };
    auto copy_sb = [&](int i, int slot) Q4_INLINE {
      const int c = wid % (BN / 64);
      copy4_to_lds(rsrc(sb_at + int64_t(i) * g.sb_ld * 4, i < steps ? b_left * 4 : 0),
                   lds0 + SB + slot * (BN * 4) + c * 256, (c * 64 + lane) * 4);
    };
    // Copy `t` of those that step i, which lies in slot `sl`, begins: A1 of i + SLOTS - 1, B and A0 of
    // i + SLOTS.
    auto copy_next = [&](int i, int sl, int t) Q4_INLINE {
      const int before = sl == 0 ? SLOTS - 1 : sl - 1;
      if (t < CA) copy_a(i + SLOTS - 1, before, 1, t);
      else if (t < CA + CB) copy_b(i + SLOTS, sl, t - CA);
      else if (t < 2 * CA + CB) copy_a(i + SLOTS, sl, 0, t - CA - CB);
      else if (t == 2 * CA + CB) copy_sa(i + SLOTS, sl, before);
      else if (VECB && t == 2 * CA + CB + 1) copy_sb(i + SLOTS, sl);
    };
    static_assert(2 * CA + CB + (VECB ? 2 : 1) <= (MB / 2 + 1) * NB, "a place for each copy");
    typedef __attribute__((address_space(3))) const float* fptr;
    typedef __attribute__((address_space(3))) const f32x4_t* vptr;
    typename PA::Reader ra;
    typename PB::Reader rb;
    uint32_t rsa, rsb;
    auto read_a = [&](int a) { return ra.read(a / (MB / 2) * (A1 - A0), 16 * (a % (MB / 2))); };
    auto read_sa = [&](int a) {
      return *((fptr)(uintptr_t)rsa + (a / (MB / 2) * (S1 - S0) + 64 * (a % (MB / 2))) / 4);
    };
    auto read_b = [&](int b) { return rb.read(0, 16 * b); };
    auto read_sb = [&](int b) { return *((vptr)(uintptr_t)rsb + 4 * b); };
    // the readers from slot `sl` to the next
    auto next_slot = [&](int sl) {
      const int by = sl == SLOTS - 1 ? 1 - SLOTS : 1;
      ra.move(by * PA::BYTES), rb.move(by * PB::BYTES);
      rsa += by * HR * 4, rsb += by * BN * 4;
    };
    auto fence = [] { __builtin_amdgcn_sched_barrier(0); };

  constexpr int NEXT = 2 * CA + CB + (VECB ? 2 : 1);   // copies (of a wave) in a step
  auto begin = [&]() Q4_INLINE {
    aim();
#pragma unroll
    for (int i = -SLOTS; i < 0; ++i)
#pragma unroll
      for (int t = 0; t < NEXT; ++t) copy_next(i, i + SLOTS, t);
  };
  begin();
  for (;;) {
    const BlockScale<MODE> block(g, w, w.n0 + wn * COLS);
    ra.start(lds0 + A0, lane, wm * HW);
    rb.start(lds0, lane, wn * COLS);
    rsa = lds0 + S0 + (wm * HW + (lane & 15)) * 4, rsb = lds0 + SB + (wn * COLS + 4 * (lane >> 4)) * 4;
    f32x4_t acc[MB][NB];
#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[a][b] = f32x4_t{0, 0, 0, 0};
    float sb_next = steps > 0 ? block.at(w.s_begin) : 0.f;
    wait_barrier8<0>();   // (the last tile's stores are counted with the copies)
    const bool rows = w.m0 + wm * (BM / WM) < w.m_end;
    if (!rows) {   // no row of the wave's: it copies for the others
      for (int i = 0, sl = 0; i < steps; ++i, sl = sl == SLOTS - 1 ? 0 : sl + 1) {
        wait_barrier8<(SLOTS - 2) * NEXT>();
#pragma unroll
        for (int t = 0; t < NEXT; ++t) copy_next(i, sl, t);
      }
    } else {
    Frag fa[2], fb[NB];
    float sa[2], scale = 0.f, last = 0.f;   // of the block whose results are scaled, of the one before
    f32x4_t p[2][NB], vb[VECB ? NB : 1];   // vb: the columns' scales for the results scaled next
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      fb[b] = read_b(b);
      p[1][b] = f32x4_t{0, 0, 0, 0};
      if constexpr (VECB) vb[b] = f32x4_t{0, 0, 0, 0};
    }
    fa[0] = read_a(0), sa[0] = read_sa(0);
    int sl = 0;
    for (int i = 0; i < steps; ++i) {
      const float sbs = sb_next;
      if (i + 1 < steps) sb_next = block.at(w.s_begin + i + 1);
#pragma unroll
      for (int a = 0; a < MB; ++a) {
        const int cur = a & 1;
        fence();
        if (a == MB / 2 - 1) wait_barrier8<(SLOTS - 2) * NEXT>();
        // the next block's fragment
        if (a + 1 == MB) next_slot(sl);
        fa[1 - cur] = read_a((a + 1) % MB), sa[1 - cur] = read_sa((a + 1) % MB);
        last = scale;
        scale = VECB ? sa[cur] : sa[cur] * sbs;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          fence();
          p[cur][b] = group_product(fb[b], fa[cur]);
          if (a == MB - 1) fb[b] = read_b(b);
          const int to = a == 0 ? MB - 1 : a - 1;   // the block before (a == 0: of the step before)
          f32x4_t v = p[1 - cur][b];
          if constexpr (VECB) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] *= vb[b][e];
            if (a == 0) vb[b] = read_sb(b);   // (until here the last step's)
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[to][b][e] = __builtin_fmaf(v[e], last, acc[to][b][e]);
          if (a >= MB / 2 - 1) {
            fence();
            copy_next(i, sl, (a - (MB / 2 - 1)) * NB + b);
          }
        }
      }
      sl = sl == SLOTS - 1 ? 0 : sl + 1;
    }
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        acc[MB - 1][b][e] = __builtin_fmaf(p[1][b][e] * (VECB ? vb[b][e] : 1.f), scale, acc[MB - 1][b][e]);
    }
    wait_barrier8<0>();   // every wave's copies and reads are done: LDS is free
    const Work done = w;
    item = scalar(tiles.item(++round));
    const bool more = item < tiles.limit;
    if (more) {
      w = tiles.at(g, item);
      begin();
    }
    if (rows) {
      int lane = threadIdx.x & 63;
      asm volatile("" : "+v"(lane));
      const int64_t m = done.m0 + wm * (BM / WM), n = done.n0 + wn * COLS;
      if (MODE != FP8_DW && done.part >= 0) {
        f32x4_t* o = reinterpret_cast<f32x4_t*>(g.part) + ((int64_t(done.part) * NW + wid) * MB * NB) * 64 + lane;
#pragma unroll
        for (int a = 0; a < MB; ++a)
#pragma unroll
          for (int b = 0; b < NB; ++b) o[(a * NB + b) * 64] = acc[a][b];
      } else if (g.ksplit > 1) store_slice<MB, NB>(g, done, acc, m, n, lane);
      else if (g.dtype == 1) finish64<MODE, MB, true>(g, done, acc, m, n, lane);
      else finish64<MODE, MB, false>(g, done, acc, m, n, lane);
    }
    if (!more) return;
  }
}

// Adds the slices of the tiles whose K steps were split, in slice order: a wave per 16 rows and 64
// columns, 4 waves of the product's WM x WN per workgroup; `room`: the product's workgroups.
template <int MODE, int BM, int BN, int WM, int WN>
__global__ void __launch_bounds__(256) k_fp8_tail(Fp8Args g, uint32_t mtiles, uint32_t ntiles, uint32_t room) {
  constexpr int NW = WM * WN, MB = BM / WM / 16, NB = BN / WN / 16;
  __shared__ Span span;
  __shared__ int32_t tot[4];
  const uint32_t wgs = room / 8;
  const Tiles<MODE, 256, BM, BN> tiles(g, mtiles, ntiles, wgs, &span, tot);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  const uint32_t item = tiles.full + blockIdx.x / 8 * tiles.slices;   // the tile's first slice
  if (tiles.slices == 1 || item >= tiles.limit) return;
  const Work w = tiles.at(g, item);
  const int piece = int(blockIdx.y) * 4 + wave, wid = piece / MB, a = piece % MB;   // of NW * MB
  const int64_t m = w.m0 + wid / WN * (BM / WM) + 16 * a, n = w.n0 + wid % WN * (16 * NB);
  if (m >= w.m_end) return;
  f32x4_t acc[1][NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) acc[0][b] = f32x4_t{0, 0, 0, 0};
  for (uint32_t s = 0; s < tiles.slices; ++s) {
    const f32x4_t* p = reinterpret_cast<const f32x4_t*>(g.part) + ((int64_t(w.part + int(s) * 8) * NW + wid) * MB + a) * NB * 64 + lane;
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[0][b] += p[b * 64];
  }
  if (g.dtype == 1) finish64<MODE, 1, true>(g, w, acc, m, n, lane);
  else finish64<MODE, 1, false>(g, w, acc, m, n, lane);
}

// Adds the K slices of a split product in slice order, four columns per thread.
__global__ void __launch_bounds__(256) k_fp8_join(Fp8Args g) {
  const uint32_t quads = uint32_t((g.N + 3) / 4), i = blockIdx.x * 256 + threadIdx.x;   // (fp8_plan_us: below 2^32)
  const int64_t m = i / quads;
  if (m >= g.M) return;
  const int64_t n = int64_t(i - uint32_t(m) * quads) * 4;
  const int count = int(std::min<int64_t>(4, g.N - n));
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < g.ksplit; ++s) {
    const float* q = g.part + (int64_t(s) * g.M + m) * g.N + n;
    if (count == 4 && (g.N & 3) == 0) {
      const f32x4_t u = *reinterpret_cast<const f32x4_t*>(q);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += u[e];
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < count) v[e] += q[e];
    }
  }
  store_row<4>(g.c, g.dtype, m * g.ldc + n, v, count);
}

// Few rows (per expert): bound by reading the weights once (one row, 2048 / 16384: 8 us, 4.2 TB/s).
// A workgroup owns 16 columns of y of one expert, its 8 waves take the 128-code K steps in turn and
// feed the matrix core straight from global memory, then add their sums through LDS in wave order.
template <int RB, int MAXRB>
Q4_DEVICE void rows_product(const Fp8Args& g, const uint8_t* w, const float* ws, int64_t n0, int64_t row0, int rows,
                            f32x4_t (*sums)[MAXRB][64]) {
  constexpr int W = 8;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  const int l = lane & 15, quarter = (lane >> 4) * 16;
  const uint8_t* wp = w + std::min<int64_t>(n0 + l, g.N - 1) * g.K + quarter;
  const uint8_t* xp[RB];
  const float* sp[RB];
#pragma unroll
  for (int r = 0; r < RB; ++r) {
    const int64_t m = row0 + min(16 * r + l, rows - 1);
    xp[r] = g.a + m * g.K + quarter;
    sp[r] = g.sa + m;
  }
  f32x4_t acc[RB];
#pragma unroll
  for (int r = 0; r < RB; ++r) acc[r] = f32x4_t{0, 0, 0, 0};
  const int full = int(g.K / 128);
  const int64_t sb0 = (n0 / 128) * g.sb_ld;
  auto steps = [&](auto n_c, int s) {
    constexpr int N = decltype(n_c)::value;
    Frag fw[N], fx[N][RB];
    float sc[N][RB];
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int64_t at = int64_t(s + u * W) * 128;
      fw[u].lo = *reinterpret_cast<const u32x4_t*>(wp + at);
      fw[u].hi = *reinterpret_cast<const u32x4_t*>(wp + at + 64);
      const float sw = load_uniform(ws, sb0 + s + u * W);
#pragma unroll
      for (int r = 0; r < RB; ++r) {
        fx[u][r].lo = *reinterpret_cast<const u32x4_t*>(xp[r] + at);
        fx[u][r].hi = *reinterpret_cast<const u32x4_t*>(xp[r] + at + 64);
        sc[u][r] = sw * sp[r][(s + u * W) * g.sa_ld];
      }
    }
#pragma unroll
    for (int u = 0; u < N; ++u)
#pragma unroll
      for (int r = 0; r < RB; ++r) {
        const f32x4_t p = wide_product(fw[u], fx[u][r]);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[r][e] = __builtin_fmaf(p[e], sc[u][r], acc[r][e]);
      }
  };
  constexpr int U = MAXRB > 1 && RB <= 2 ? 2 : 1;   // steps in flight
  int s = wave;
  for (; s + (U - 1) * W < full; s += U * W) steps(std::integral_constant<int, U>{}, s);
  for (; s < full; s += W) steps(std::integral_constant<int, 1>{}, s);
  if (s == full && g.K % 128) {   // the K tail: chunks past the row's end hold zeros
    const int64_t at = int64_t(full) * 128;
    const bool lo = at + quarter < g.K, hi = at + 64 + quarter < g.K;
    const u32x4_t zero = {0, 0, 0, 0};
    Frag fw;
    fw.lo = lo ? *reinterpret_cast<const u32x4_t*>(wp + at) : zero;
    fw.hi = hi ? *reinterpret_cast<const u32x4_t*>(wp + at + 64) : zero;
    const float sw = load_uniform(ws, sb0 + full);
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      Frag fx;
      fx.lo = lo ? *reinterpret_cast<const u32x4_t*>(xp[r] + at) : zero;
      fx.hi = hi ? *reinterpret_cast<const u32x4_t*>(xp[r] + at + 64) : zero;
      const float sc = sw * sp[r][full * g.sa_ld];
      const f32x4_t p = wide_product(fw, fx);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[r][e] = __builtin_fmaf(p[e], sc, acc[r][e]);
    }
  }
#pragma unroll
  for (int r = 0; r < RB; ++r) sums[wave][r][lane] = acc[r];
  __syncthreads();
  if (wave < RB) {
    f32x4_t v = sums[0][wave][lane];
#pragma unroll
    for (int i = 1; i < W; ++i) v += sums[i][wave][lane];
    const int m = 16 * wave + l;
    const int64_t n = n0 + 4 * (lane >> 4);
    const float o[4] = {v[0], v[1], v[2], v[3]};
    if (m < rows && n < g.N)
      store_row<4>(g.c, g.dtype, (row0 + m) * g.ldc + n, o, int(std::min<int64_t>(4, g.N - n)));
  }
  __syncthreads();
}

// The expert with the i-th of the runs of rows that are not empty, or -1: all of a workgroup's 8
// waves call, 64 experts each at a time.
Q4_DEVICE int nth_run(const int32_t* offsets, int e, int64_t t, int i, uint64_t* runs /* LDS [8] */) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  for (int x0 = 0; x0 < e; x0 += 512) {
    int64_t first, count = 0;
    if (x0 + int(threadIdx.x) < e) expert_rows(offsets, x0 + int(threadIdx.x), t, first, count);
    const uint64_t own = __ballot(count > 0);
    if (lane == 0) runs[wave] = own;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const uint64_t m = scalar(runs[w]);
      const int n = __popcll(m);
      if (i < n) {
        const bool mine = (m >> lane & 1) && __popcll(m & ((uint64_t(1) << lane) - 1)) == i;
        return scalar(x0 + 64 * w + __ffsll((unsigned long long)__ballot(mine)) - 1);
      }
      i -= n;
    }
    __syncthreads();
  }
  return -1;
}

// Workgroup (x, n): 16 columns of expert x; with `search`, of the x-th expert that has a row.
template <int MAXRB>
__global__ void __launch_bounds__(512) k_fp8_rows(Fp8Args g, uint32_t ncols, int search) {
  __shared__ f32x4_t sums[8][MAXRB][64];
  __shared__ uint64_t runs[8];
  int x = int(blockIdx.x / ncols);
  const int64_t n0 = int64_t(blockIdx.x - x * ncols) * 16;
  if (search) x = nth_run(g.offsets, g.e, g.M, x, runs);
  if (x < 0) return;
  int64_t first = 0, count = g.M;
  if (g.offsets) expert_rows(g.offsets, x, g.M, first, count);
  const uint8_t* w = g.b + x * g.b_stride;
  const float* ws = g.sb + x * g.sb_stride;
  while (count > 0) {
    const int rows = int(count < 16 * MAXRB ? count : 16 * MAXRB);
    if constexpr (MAXRB == 1) {
      rows_product<1, 1>(g, w, ws, n0, first, rows, sums);
    } else {
      if (rows <= 16) rows_product<1, MAXRB>(g, w, ws, n0, first, rows, sums);
      else if (rows <= 32) rows_product<2, MAXRB>(g, w, ws, n0, first, rows, sums);
      else rows_product<MAXRB, MAXRB>(g, w, ws, n0, first, rows, sums);
    }
    first += rows, count -= rows;
  }
}

// Passes of 16 rows with one step in flight per wave and as many waves as fit (four steps in flight
// of fewer waves: one row, 8192 / 8192, 16.6 -> 17 us, 4096 / 14336 15.7 -> 17, 16 rows of 8192 / 8192
// 21 -> 23, 64 rows of 32 experts, 7168 / 4096, 143 -> 166), or of 64 with two (8 to 32 rows of 32
// experts, 16384 / 256, 38 us; with one 41).
hipError_t launch_rows8(const Fp8Args& g, bool few, hipStream_t st) {
  const uint32_t ncols = uint32_t(ceil_div(g.N, 16));
  const int64_t e = g.offsets ? g.e : 1;
  const bool search = fp8_rows_search(g.M, g.N, e);   // (never with one)
  const dim3 grid(unsigned(fp8_rows_grid(g.M, g.N, e)));
  if (few) hipLaunchKernelGGL((k_fp8_rows<1>), grid, dim3(512), 0, st, g, ncols, search);
  else hipLaunchKernelGGL((k_fp8_rows<4>), grid, dim3(512), 0, st, g, ncols, search);
  return hipGetLastError();
}

// ---------------------------------------------------------------- launches
template <int MODE>
hipError_t launch_tiles8(Fp8Args g, const Plan& p, hipStream_t st) {
  g.ksplit = p.ksplit;
  g.tail = fp8_has_tail(p, Fp8Mode(MODE), ceil_div(g.K, 128), g.offsets != nullptr);
  const uint32_t nt = uint32_t(ceil_div(g.N, p.tile));
  uint32_t mt = uint32_t(ceil_div(g.M, p.tile));
  int64_t items;
  if (MODE != FP8_DW && g.offsets)   // as many tiles as the offsets can make
    items = (g.M / p.tile + std::min<int64_t>(g.e, g.M)) * nt;
  else items = int64_t(mt) * nt * (MODE == FP8_DW ? g.e : 1) * p.ksplit;
  // (the large tiles' workgroups, as many as the card holds, walk their tiles; so do all by expert)
  unsigned grid = unsigned(items);
  if (p.tile != 64 || (MODE != FP8_DW && g.offsets)) {
    const int64_t room = 256 * (p.tile == 256 ? 1 : p.tile == 128 ? 2 : 3);
    grid = unsigned(g.tail ? room : std::min<int64_t>(room, ceil_div(items, 8) * 8));
  }
  if (p.tile == 256) hipLaunchKernelGGL((k_fp8_big<MODE, 256, 256, 2, 4, 2>), dim3(grid), dim3(512), 0, st, g, mt, nt);
  else if (p.tile == 128) hipLaunchKernelGGL((k_fp8_big<MODE, 128, 128, 2, 2, 2>), dim3(grid), dim3(256), 0, st, g, mt, nt);
  else hipLaunchKernelGGL((k_fp8<MODE, 64, 64, 2, 2, 3>), dim3(grid), dim3(256), 0, st, g, mt, nt);
  const hipError_t e = hipGetLastError();
  if constexpr (MODE != FP8_DW)
    if (e == hipSuccess && g.tail) {   // (at most half of an XCD's workgroups have a tile to split)
      if (p.tile == 256) hipLaunchKernelGGL((k_fp8_tail<MODE, 256, 256, 2, 4>), dim3(grid / 2, 16), dim3(256), 0, st, g, mt, nt, grid);
      else hipLaunchKernelGGL((k_fp8_tail<MODE, 128, 128, 2, 2>), dim3(grid / 2, 4), dim3(256), 0, st, g, mt, nt, grid);
      return hipGetLastError();
    }
  if (e != hipSuccess || p.ksplit == 1) return e;
  const int64_t threads = g.M * ((g.N + 3) / 4);
  hipLaunchKernelGGL(k_fp8_join, dim3(unsigned(ceil_div(threads, 256))), dim3(256), 0, st, g);
  return hipGetLastError();
}

int64_t part_bytes8(const Plan& p, Fp8Mode mode, int64_t m, int64_t n, int64_t steps, bool grouped) {
  if (fp8_has_tail(p, mode, steps, grouped)) return int64_t(256) * (p.tile == 256 ? 1 : 2) * p.tile * p.tile * 4;
  return p.ksplit > 1 ? int64_t(p.ksplit) * m * n * 4 : 0;
}

template <int DT>
hipError_t quantize_as(const Fp8QuantArgs& a, hipStream_t st) {
  const bool rows = a.q_row, cols = a.q_col;
  const int64_t tiles = cols && a.offsets ? a.t / 128 + std::min<int64_t>(a.e, a.t) : ceil_div(a.t, cols ? 128 : 16 * kRowsAlone);
  const dim3 grid(unsigned(tiles), unsigned(ceil_div(a.k, 128)));
  auto go = [&](auto kern) { hipLaunchKernelGGL(kern, grid, dim3(256), 0, st, a); };
  if (a.gated) go(k_quantize_fp8<DT, FORM_ROWS, true>);
  else if (rows && cols) go(k_quantize_fp8<DT, FORM_ROWS | FORM_COLS, false>);
  else if (cols) go(k_quantize_fp8<DT, FORM_COLS, false>);
  else go(k_quantize_fp8<DT, FORM_ROWS, false>);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_fp8_tokens(const Fp8QuantArgs& a, hipStream_t st) {
  return a.dtype == 0 ? quantize_as<0>(a, st) : a.dtype == 1 ? quantize_as<1>(a, st) : quantize_as<2>(a, st);
}

hipError_t launch_quantize_fp8_blocks(const void* w, int dtype, int64_t e, int64_t n, int64_t k, uint8_t* q, float* s,
                                      hipStream_t st) {
  const uint32_t rb = uint32_t(ceil_div(n, 128));
  const dim3 grid(unsigned(e * rb), unsigned(ceil_div(k, 128)));
  auto go = [&](auto kern) { hipLaunchKernelGGL(kern, grid, dim3(256), 0, st, w, n, k, rb, q, s); };
  if (dtype == 0) go(k_quantize_fp8_blocks<0>);
  else if (dtype == 1) go(k_quantize_fp8_blocks<1>);
  else go(k_quantize_fp8_blocks<2>);
  return hipGetLastError();
}

int64_t fp8_linear_workspace(int64_t t, int64_t k, int64_t n, int32_t e, bool grouped) {
  return t == 0 ? 0 : part_bytes8(fp8_plan(FP8_Y, t, k, n, e, grouped), FP8_Y, t, n, ceil_div(k, 128), grouped);
}

hipError_t launch_fp8_linear(const uint8_t* q, const float* s, int64_t t, int64_t k, const uint8_t* wq, const float* ws,
                             int64_t n, const int32_t* offsets, int32_t e, int y_dtype, void* y, void* work,
                             hipStream_t st) {
  Fp8Args g{};
  g.a = q, g.b = wq;
  g.lda = g.ldb = k;
  g.sa = s, g.sb = ws;
  g.sa_ld = t, g.sb_ld = ceil_div(k, 128);
  g.M = t, g.N = n, g.K = k;
  g.b_stride = n * k, g.sb_stride = ceil_div(n, 128) * g.sb_ld;
  g.offsets = offsets, g.e = e;
  g.dtype = y_dtype;
  g.c = y, g.ldc = n;
  g.ksplit = 1;
  g.part = static_cast<float*>(work);
  const Plan p = fp8_plan(FP8_Y, t, k, n, e, offsets != nullptr);
  if (p.tile) return launch_tiles8<FP8_Y>(g, p, st);
  return launch_rows8(g, fp8_rows_sixteen(t, e, offsets != nullptr), st);
}

// Workspace of the gradients: codes and scales of dy along its rows and along the tokens, the K
// slices of whichever product splits K.
struct Fp8GradWork {
  Plan dx, dw;
  uint8_t *q_row, *q_col;
  float *s_row, *s_col, *part;
  int64_t bytes;
};
static Fp8GradWork grad_work8(void* base, int64_t t, int64_t k, int64_t n, int32_t e, bool grouped) {
  Fp8GradWork w{};
  w.dx = fp8_plan(FP8_DX, t, k, n, e, grouped);
  w.dw = fp8_plan(FP8_DW, t, k, n, e, grouped);
  auto take = [&](int64_t bytes) {
    uint8_t* p = static_cast<uint8_t*>(base) + w.bytes;
    w.bytes += align256(bytes);
    return p;
  };
  w.q_row = take(t * n), w.q_col = take(t * n);
  w.s_row = reinterpret_cast<float*>(take(ceil_div(n, 128) * t * 4));
  w.s_col = reinterpret_cast<float*>(take((grouped ? t / 128 + std::min<int64_t>(e, t) : ceil_div(t, 128)) * n * 4));
  w.part = reinterpret_cast<float*>(take(std::max(part_bytes8(w.dx, FP8_DX, t, k, ceil_div(n, 128), grouped),
                                                      part_bytes8(w.dw, FP8_DW, n, k, 0, grouped))));
  return w;
}
int64_t fp8_linear_bwd_workspace(int64_t t, int64_t k, int64_t n, int32_t e, bool grouped) {
  return t == 0 ? 0 : grad_work8(nullptr, t, k, n, e, grouped).bytes;
}

hipError_t launch_fp8_linear_bwd(const void* dy, int64_t t, int64_t k, int64_t n, int dtype, const uint8_t* xq,
                                 const float* xs, const uint8_t* wq, const float* ws, const int32_t* offsets, int32_t e,
                                 void* dx, void* dw, void* work, hipStream_t st) {
  const bool grouped = offsets != nullptr;
  const Fp8GradWork w = grad_work8(work, t, k, n, e, grouped);
  Fp8Args g{};
  g.dtype = dtype;
  g.ksplit = 1;
  g.part = w.part;
  g.offsets = offsets, g.e = e;
  if (t > 0) {
    const Fp8QuantArgs a{dy, t, n, dtype, 0, w.q_row, w.q_col, w.s_row, w.s_col, offsets, e};
    hipError_t rc = launch_quantize_fp8_tokens(a, st);
    if (rc != hipSuccess) return rc;
    g.a = w.q_row, g.b = wq;
    g.lda = n, g.ldb = k;
    g.sa = w.s_row, g.sb = ws;
    g.sa_ld = t, g.sb_ld = ceil_div(k, 128);
    g.M = t, g.N = k, g.K = n;
    g.b_stride = n * k, g.sb_stride = ceil_div(n, 128) * g.sb_ld;
    g.c = dx, g.ldc = k;
    rc = launch_tiles8<FP8_DX>(g, w.dx, st);
    if (rc != hipSuccess) return rc;
  }
  g.a = w.q_col, g.b = xq;   // (t == 0: no K step, zeros)
  g.lda = n, g.ldb = k;
  g.sa = w.s_col, g.sb = xs;
  g.sa_ld = n, g.sb_ld = k;
  g.M = n, g.N = k, g.K = t;
  g.b_stride = g.sb_stride = 0;
  g.c = dw, g.ldc = k;
  return launch_tiles8<FP8_DW>(g, w.dw, st);
}

}  // namespace q4
