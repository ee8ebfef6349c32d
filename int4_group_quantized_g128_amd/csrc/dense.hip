// Dense products on the matrix cores: the INT8 linear with a scale per token and per
// output channel, and the 16-bit gated projection with its gradients.
//
//   int8    y[t][n]  = (sum_k q[t][k] wq[n][k]) * (s[t] ws[n]) + b[n]
//   swiglu  h        = silu(g) * u,  g = x Wg^T,  u = x Wu^T
//   grads   dg = dh u sig(g) (1 + g (1 - sig(g))),  du = dh silu(g)
//           dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x
//
// Operands are read as they lie in memory: "KC" panels are contiguous along K (x, q and
// the weights of the forward products), "MC" panels along their own row index (the
// weights in dx; dg, du and x in the weight gradients), whose fragments come out of LDS
// through the transposing 8-byte reads, so no transposed copy is ever made.
//
// Tiles: K advances SB = 64 or 128 bytes per step (32 to 128 elements).  Panels are copied
// global -> LDS in 16-byte chunks; the buffer descriptor of each step covers exactly what
// is left of the panel, so rows past its end and the masked K tail read as zero.  Chunks
// are XOR-swizzled so that the fragment reads hit distinct banks:
//   KC  [rows][SB]: chunk c of row r at c ^ f(r), f over the rows that share a bank period
//   MC  [K of a step][2 rows B]: 32-byte piece p of row k at p ^ f(k), f from the bits of k
//       that differ between the 8 rows a transposing read touches at once.
#include <type_traits>

#include "common.h"
#include "dense.h"
#include "dense_plan.h"
#include "internal.h"
#include "lds_copy.h"

namespace q4 {

namespace {

constexpr int kStepBytes = 128;
constexpr uint32_t kNoByte = 0x80000000u;   // a byte offset past every descriptor's range

// SCALED: as STORE, each row times its own power of two.
enum Epi { EPI_STORE = 0, EPI_SWIGLU = 1, EPI_INT8 = 2, EPI_SCALED = 3 };
constexpr bool row_scaled(int epi) { return epi == EPI_INT8 || epi == EPI_SCALED; }

template <Act A> struct Num {
  static constexpr int ESZ = A == Act::I8 ? 1 : 2;
  typedef typename std::conditional<A == Act::I8, i32x4_t, f32x4_t>::type acc_t;
  static Q4_DEVICE acc_t mfma(u32x4_t a, u32x4_t b, acc_t c) {
    if constexpr (A == Act::I8) return mfma_i8_16x16x64(a, b, c);
    else return mfma16x16x32<A>(a, b, c);
  }
};

// One product C[m][n] = sum_k A(m, k) B(n, k), possibly over two K segments (a[s], b[s]),
// for two batches (a[z], c[z]) or with two B panels side by side (swiglu: b[0], b[1]).
struct DenseArgs {
  const void* a[2];
  const void* b[2];
  int64_t lda, ldb;
  int32_t M, N, K;
  int32_t batches, ksplit;
  void* c[2];
  int64_t ldc;
  int32_t c_dtype;          // 0 fp32, 1 fp16, 2 bf16
  const float* s_row;       // int8: token scales; scaled: [batches][M]
  const float* s_col;       // int8: channel scales
  const float* bias;        // int8: or NULL
  float* gu;                // swiglu: [M][2][N] products, or NULL
  void* part;               // ksplit > 1: [ksplit][batches][panels][M][N] fp32 / int32 sums
};

Q4_DEVICE uint16_t to16(float v, int dtype) {
  return dtype == 1 ? bitcast<uint16_t>(_Float16(v)) : bitcast<uint16_t>(__bf16(v));
}

// Stores up to four consecutive values of a row.
Q4_DEVICE void store4(void* c, int dtype, int64_t idx, f32x4_t v, int count, bool vec) {
  if (dtype == 0) {
    float* p = static_cast<float*>(c) + idx;
    if (vec && count == 4) {
      *reinterpret_cast<f32x4_t*>(p) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < count) p[i] = v[i];
    }
  } else {
    uint16_t* p = static_cast<uint16_t*>(c) + idx;
    uint16_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = to16(v[i], dtype);
    if (vec && count == 4) {
      *reinterpret_cast<uint2*>(p) = make_uint2(h[0] | uint32_t(h[1]) << 16, h[2] | uint32_t(h[3]) << 16);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < count) p[i] = h[i];
    }
  }
}

// Channel scales and bias of four columns n .. n + 3.
struct ColScales {
  f32x4_t s, b;
};
template <int EPI>
Q4_DEVICE ColScales col_scales(const DenseArgs& g, int n) {
  ColScales r;
  if constexpr (EPI == EPI_INT8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = min(n + i, g.N - 1);
      r.s[i] = g.s_col[c];
      r.b[i] = g.bias ? g.bias[c] : 0.f;
    }
  }
  return r;
}
template <int EPI>
Q4_DEVICE float row_scale(const DenseArgs& g, int z, int m) {
  if constexpr (row_scaled(EPI)) return g.s_row[(EPI == EPI_SCALED ? int64_t(z) * g.M : 0) + min(m, g.M - 1)];
  return 0.f;
}

// Four values of the result from the sums v (v2: the second B panel's).
template <Act A, int EPI>
Q4_DEVICE f32x4_t result4(typename Num<A>::acc_t v, typename Num<A>::acc_t v2, float sm, const ColScales& cs) {
  f32x4_t y;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // int8: the INT32 sum becomes fp32 (24 bits), the scales' product is rounded, and one fma
    // joins them and the bias (spelt out, so that every kernel rounds alike)
    if constexpr (EPI == EPI_INT8) y[i] = __builtin_fmaf(float(v[i]), sm * cs.s[i], cs.b[i]);
    else if constexpr (EPI == EPI_SWIGLU) y[i] = swiglu(v[i], v2[i]);
    else if constexpr (EPI == EPI_SCALED) y[i] = v[i] * sm;
    else y[i] = v[i];
  }
  return y;
}

// Result of four columns n .. n + 3 of row m.
template <Act A, int EPI>
Q4_DEVICE void finish4(const DenseArgs& g, int z, int m, int n, typename Num<A>::acc_t v, typename Num<A>::acc_t v2,
                       float sm, const ColScales& cs) {
  if (m >= g.M || n >= g.N) return;
  const int count = min(4, g.N - n);
  const bool vec = (g.ldc & 3) == 0;
  store4(z ? g.c[1] : g.c[0], g.c_dtype, int64_t(m) * g.ldc + n, result4<A, EPI>(v, v2, sm, cs), count, vec);
  if constexpr (EPI == EPI_SWIGLU) {
    if (g.gu) {
      const int64_t at = int64_t(m) * 2 * g.ldc + n;
      store4(g.gu, 0, at, v, count, vec);
      store4(g.gu, 0, at + g.ldc, v2, count, vec);
    }
  }
}

// Raw sums of a K slice, columns n .. n + 3.
template <typename V>
Q4_DEVICE void store_part(const DenseArgs& g, int64_t panel, int m, int n, V v) {
  uint32_t* o = static_cast<uint32_t*>(g.part) + (panel * g.M + m) * g.N + n;
  const u32x4_t w = bitcast<u32x4_t>(v);
  if (n + 4 <= g.N && (g.N & 3) == 0) {
    *reinterpret_cast<u32x4_t*>(o) = w;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < g.N) o[e] = w[e];
  }
}

// Eight consecutive 16-bit values of a row (8 lanes: a whole 128-byte line).  NT: written past
// the caches' reuse order, which the gradients gain from (backward 524 -> 513 us at 4096 x 2048 x
// 8192) and INT8 results do not (76.0 -> 78.5 us at 2048 x 2048 x 16384).
template <bool NT>
Q4_DEVICE void store8(void* c, int dtype, int64_t idx, f32x4_t y0, f32x4_t y1, int count, int64_t ld) {
  if (dtype != 0 && count >= 8 && (ld & 7) == 0) {
    u32x4_t o;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      o[w] = to16(y0[2 * w], dtype) | uint32_t(to16(y0[2 * w + 1], dtype)) << 16;
      o[2 + w] = to16(y1[2 * w], dtype) | uint32_t(to16(y1[2 * w + 1], dtype)) << 16;
    }
    u32x4_t* p = reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(c) + idx);
    if constexpr (NT) __builtin_nontemporal_store(o, p);
    else *p = o;
  } else {
    const bool vec = (ld & 3) == 0;
    store4(c, dtype, idx, y0, min(count, 4), vec);
    store4(c, dtype, idx + 4, y1, min(count - 4, 4), vec);
  }
}

// The end of a tile: a wave's sums go through its own part of LDS (free once every wave's
// copies are done), 64 fp32 columns (or 32) per row, so that a lane holds 8 consecutive
// columns of one row, or 4 of both projections, stores are whole lines, and the code that
// turns sums into results stands in one short loop (stored from the accumulators it was 30 KB
// of code: forward with g and u 277 -> 270 us at 4096 x 2048 x 8192).
// 16-byte chunk c of row r lies at c ^ (r % chunks of a row), against bank conflicts.
template <int COLS, typename V>
Q4_DEVICE void turn_in(uint32_t lds, int row, int chunk, V v) {
  typedef __attribute__((address_space(3))) V* lptr;
  constexpr int CH = COLS / 4;
  *(lptr)(uintptr_t)(lds + row * (COLS * 4) + ((chunk ^ (row & (CH - 1))) << 4)) = v;
}

template <Act A, int EPI, int COLS>
Q4_DEVICE void turn_out(const DenseArgs& g, int z, int64_t slice, uint32_t lds, int lane, int rows, int m0, int n0,
                        const float* s_row) {
  typedef typename Num<A>::acc_t acc_t;
  typedef __attribute__((address_space(3))) const acc_t* lptr;
  constexpr bool DUAL = EPI == EPI_SWIGLU;
  constexpr int CH = COLS / 4, LPR = COLS / 8;   // chunks and lanes per row
  const int c = lane % LPR, n = n0 + (DUAL ? 4 : 8) * c;
  const int ca = DUAL ? c : 2 * c, cb = DUAL ? CH / 2 + c : 2 * c + 1;
  const ColScales cs0 = col_scales<EPI>(g, n), cs1 = col_scales<EPI>(g, n + 4);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // other lanes' turn_in before these reads
#pragma unroll 2
  for (int r = lane / LPR; r < rows; r += 64 / LPR) {
    const acc_t a = *(lptr)(uintptr_t)(lds + r * (COLS * 4) + ((ca ^ (r & (CH - 1))) << 4));
    const acc_t b = *(lptr)(uintptr_t)(lds + r * (COLS * 4) + ((cb ^ (r & (CH - 1))) << 4));
    const int m = m0 + r;
    if (m >= g.M || n >= g.N) continue;
    if (g.ksplit > 1) {
      store_part(g, DUAL ? 2 * slice : slice, m, n, a);
      if (DUAL) store_part(g, 2 * slice + 1, m, n, b);
      else if (n + 4 < g.N) store_part(g, slice, m, n + 4, b);
      continue;
    }
    if constexpr (DUAL) {
      const int64_t at = int64_t(m) * g.ldc + n;   // (ldc is a multiple of 8: whole quads)
      store4(g.c[0], g.c_dtype, at, result4<A, EPI>(a, b, 0.f, cs0), 4, true);
      if (g.gu) {
        // (past the caches a forward alone gains 20 us of 300 at 4096 x 2048 x 8192, but a backward
        // pass that follows it at once loses 57: 796 -> 833 us for both)
        f32x4_t* p = reinterpret_cast<f32x4_t*>(g.gu + at + int64_t(m) * g.ldc);
        *p = a;
        *(p + g.ldc / 4) = b;
      }
    } else {
      const float sm = row_scaled(EPI) ? s_row[r] : 0.f;
      store8<EPI != EPI_INT8>(z ? g.c[1] : g.c[0], g.c_dtype, int64_t(m) * g.ldc + n, result4<A, EPI>(a, a, sm, cs0),
             result4<A, EPI>(b, b, sm, cs1), g.N - n, g.ldc);
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // these reads before the next turn_in
}

// ---------------------------------------------------------------- panels in LDS
// R rows of one operand, one K step of SB bytes: SB R bytes in copies of 1 KB.
template <Act A, bool MC, int R, int SB>
struct Panel {
  static_assert(!MC || A != Act::I8, "transposing reads are for 16-bit values");
  static constexpr int BYTES = R * SB;
  static constexpr int COPIES = BYTES / 1024;
  static constexpr int ESZ = Num<A>::ESZ;
  static constexpr int CPR = MC ? R / 8 : SB / 16;   // 16-byte chunks per LDS row

  static Q4_DEVICE int swz(int r) {
    if constexpr (!MC) return SB == 128 ? (r >> 1) & 7 : -(r >> 2) & 3;
    else if constexpr (R >= 128) return (r & 3) | ((r >> 3) & 1) << 2;
    else return ((r >> 1) & 1) | ((r >> 3) & 1) << 1;
  }

  // Lane's place in copy `copy`: LDS row and the global chunk that lands in its slot.
  static Q4_DEVICE void place(int copy, int lane, int& r, int& c) {
    const int id = copy * 64 + lane;
    r = id / CPR;
    const int slot = id % CPR;
    c = MC ? (((slot >> 1) ^ swz(r)) << 1 | (slot & 1)) : slot ^ swz(r);
  }

  // Byte offset of the lane's chunk from the panel's (first row, first k of the step).
  // `left`: KC, bytes of K left at the step; MC, columns left at the first column.
  static Q4_DEVICE uint32_t offset(int copy, int lane, int64_t ld, int left) {
    int r, c;
    place(copy, lane, r, c);
    const bool in = MC ? c * 8 < left : c * 16 < left;
    return in ? uint32_t(r * ld * ESZ + c * 16) : kNoByte;
  }

  // What is left of the panel from the next K step on: `left` bytes at `addr`; a step
  // advances by `inc` bytes.
  struct Feed {
    uint64_t addr, left;
    uint32_t inc;
    Q4_DEVICE u32x4_t rsrc(bool valid) const {   // empty if !valid
      const uint32_t high = uint32_t(left >> 32) | uint32_t(left) >> 31;
      return u32x4_t{uint32_t(addr), uint32_t(addr >> 32) & 0xffffu,
                     !valid ? 0u : high ? 0x7fffffffu : uint32_t(left), 0x00020000u};
    }
    Q4_DEVICE void next() { addr += inc, left -= inc; }
  };
  // The panel from row `row0` on (rows x K elements, leading dimension ld), at step `step`.
  static Q4_DEVICE Feed feed(const void* p, int64_t ld, int rows, int K, int row0, int step) {
    const uint32_t inc = MC ? uint32_t(ld) * SB : uint32_t(SB);
    const uint64_t at = uint64_t(MC ? int64_t(row0) : int64_t(row0) * ld) * ESZ + uint64_t(uint32_t(step)) * inc;
    return Feed{reinterpret_cast<uint64_t>(p) + at, uint64_t(MC ? int64_t(K) * ld : int64_t(rows) * ld) * ESZ - at, inc};
  }

  // Lane's byte address of a fragment read at block 0, half 0; blocks and halves flip bits
  // or add constants (the swizzle depends on lane bits only).
  static Q4_DEVICE uint32_t lane_base(int lane) {
    if constexpr (!MC) {
      const int r = lane & 15;
      return r * SB + (((lane >> 4) ^ swz(r)) << 4);
    } else {
      const int k = 8 * (lane >> 4) + ((lane & 15) >> 2);
      return k * (2 * R) + (swz(k) << 5) + ((lane & 3) << 3);
    }
  }
  // Fragment of rows r0 .. r0 + 15 (r0 % 16 == 0), half `sub` of the step: lane (row
  // lane % 16, quarter lane / 16) holds 16 bytes of K, quarter-major.  lds: the panel's LDS
  // byte address (a multiple of 1024), lb: lane_base.
  static Q4_DEVICE u32x4_t frag(uint32_t lds, uint32_t lb, int r0, int sub) {
    if constexpr (!MC) {
      typedef __attribute__((address_space(3))) const u32x4_t* lptr;
      return *(lptr)(uintptr_t)(lds + r0 * SB + (lb ^ (sub << 6)));
    } else {
      typedef short s16x4 __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) s16x4* lptr;
      const uint32_t at = lds + sub * 32 * (2 * R) + (lb ^ ((r0 >> 4) << 5));
      const u32x2_t a = bitcast<u32x2_t>(__builtin_amdgcn_ds_read_tr16_b64_v4i16((lptr)(uintptr_t)(at)));
      const u32x2_t b = bitcast<u32x2_t>(__builtin_amdgcn_ds_read_tr16_b64_v4i16((lptr)(uintptr_t)(at + 4 * (2 * R))));
      return u32x4_t{a[0], a[1], b[0], b[1]};
    }
  }
};

// Copies first .. first + N - 1 of a panel's K step into its LDS image at `at`.
template <typename P, int N>
Q4_DEVICE void copies(const u32x4_t& rs, uint32_t at, int first, int lane, int64_t ld, int left) {
  if constexpr (N == 2) {
    copy2_to_lds(rs, at + first * 1024, P::offset(first, lane, ld, left), P::offset(first + 1, lane, ld, left));
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) copy_to_lds(rs, at + (first + j) * 1024, P::offset(first + j, lane, ld, left));
  }
}

// Waits until at most N copies of this wave are in flight and its LDS reads are done,
// then joins the workgroup's barrier.
template <int N>
Q4_DEVICE void wait_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// K segments of a product: dx (the one of a KC and an MC panel) runs over the gate rows, then
// over the up rows; the others have one.
constexpr int segments(bool amc, bool bmc) { return !amc && bmc ? 2 : 1; }

// Work item of a workgroup: workgroup b runs on XCD b % 8; each XCD takes one contiguous
// range of items (its L2 keeps the panels they share), in groups of 8 row tiles that walk
// the column tiles together.
struct Item {
  int z, ks, mt, nt;
};
Q4_DEVICE Item item_of(uint32_t b, uint32_t total, uint32_t batches, uint32_t mtiles, uint32_t ntiles) {
  const uint32_t xcd = b % 8, per = total / 8, rest = total % 8;
  uint32_t i = xcd * per + (xcd < rest ? xcd : rest) + b / 8;
  Item it;
  const uint32_t tiles = mtiles * ntiles;   // (total, and so every product here, is below 2^31)
  it.ks = int(i / (tiles * batches));
  i -= it.ks * tiles * batches;
  it.z = int(i / tiles);
  i -= it.z * tiles;
  constexpr uint32_t GM = 8;
  const uint32_t band = i / (GM * ntiles);
  const uint32_t m0 = band * GM, gm = mtiles - m0 < GM ? mtiles - m0 : GM;
  i -= band * GM * ntiles;
  it.mt = int(m0 + i % gm);
  it.nt = int(i / gm);
  return it;
}

// ---------------------------------------------------------------- tile kernel
// BM x BN per workgroup of 2 x 2 waves, a ring of NS K steps of SB bytes in LDS: step
// s + NS - 1 is copied while step s is multiplied, one barrier per step.  128 x 128 tiles
// take 4 x 64 bytes (64 KB, two workgroups per CU, each hiding the other's barriers), 64 x 64
// tiles 3 x 128 bytes (48 KB, three per CU).
template <Act A, bool AMC, bool BMC, int BM, int BN, int SB, int NS, int EPI>
__global__ void __launch_bounds__(256) k_dense(DenseArgs g, int mtiles, int ntiles) {
  typedef Num<A> T;
  typedef typename T::acc_t acc_t;
  constexpr bool DUAL = EPI == EPI_SWIGLU;
  constexpr int SEGS = segments(AMC, BMC);
  constexpr int BP = DUAL ? BN / 2 : BN;            // rows of a B panel
  typedef Panel<A, AMC, BM, SB> PA;
  typedef Panel<A, BMC, BP, SB> PB;
  constexpr int STEP = SB / T::ESZ;                 // K elements per step
  constexpr int NP = DUAL ? 2 : 1;
  constexpr int STAGE = PA::BYTES + NP * PB::BYTES;
  constexpr int CA = PA::COPIES / 4, CB = PB::COPIES / 4;   // copies per wave
  constexpr int CPW = CA + NP * CB;
  constexpr int MB = BM / 32, NB = BP / 32;         // 16-blocks per wave
  __shared__ __align__(16) uint8_t ring[NS * STAGE];

  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  const int wm = wid & 1, wn = wid >> 1;
  const Item it = item_of(blockIdx.x, gridDim.x, g.batches, mtiles, ntiles);
  const int m0 = it.mt * BM, n0 = it.nt * BP;
  const int seg_steps = (g.K + STEP - 1) / STEP;
  const int all = seg_steps * SEGS;
  const int per = (all + g.ksplit - 1) / g.ksplit;
  const int s_begin = it.ks * per, s_end = min(all, s_begin + per);

  const uint32_t lds0 = lds_addr(ring);
  // the next step to copy: its place in each panel, its bytes of K, its slot
  int si = s_begin, k_left = g.K * T::ESZ, slot_in = 0;
  typename PA::Feed fda;
  typename PB::Feed fdb[NP];
  auto start = [&](int seg, int step) {
    fda = PA::feed((SEGS == 2 ? seg : it.z) ? g.a[1] : g.a[0], g.lda, g.M, g.K, m0, step);
#pragma unroll
    for (int p = 0; p < NP; ++p)
      fdb[p] = PB::feed((DUAL ? p : seg) ? g.b[1] : g.b[0], g.ldb, g.N, g.K, n0, step);
    k_left = g.K * T::ESZ - step * SB;
  };
  if (SEGS == 1 || s_begin < seg_steps) start(0, s_begin);
  else start(1, s_begin - seg_steps);
  auto issue = [&]() {
    if constexpr (SEGS == 2)
      if (si == seg_steps) start(1, 0);
    const bool in = si < s_end;
    const uint32_t at = lds0 + slot_in * STAGE;
    copies<PA, CA>(fda.rsrc(in), at, wid * CA, lane, g.lda, AMC ? g.M - m0 : k_left);
    fda.next();
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      copies<PB, CB>(fdb[p].rsrc(in), at + PA::BYTES + p * PB::BYTES, wid * CB, lane, g.ldb, BMC ? g.N - n0 : k_left);
      fdb[p].next();
    }
    k_left -= SB;
    ++si;
    slot_in = slot_in == NS - 1 ? 0 : slot_in + 1;
  };
  const uint32_t lba = PA::lane_base(lane), lbb = PB::lane_base(lane);

  acc_t acc[NP][MB][NB];
#pragma unroll
  for (int p = 0; p < NP; ++p)
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[p][i][j] = acc_t{0, 0, 0, 0};

  constexpr int AHEAD = NS - 1;   // steps in flight beyond the current one's
#pragma unroll
  for (int a = 0; a < AHEAD; ++a) issue();
  int slot = 0;
  for (int s = s_begin; s < s_end; ++s) {
    // step s is in LDS for every wave, and every wave is done reading step s - 1
    wait_barrier<(AHEAD - 1) * CPW>();
    const uint32_t base = lds0 + slot * STAGE;
    slot = slot == NS - 1 ? 0 : slot + 1;
    u32x4_t fa[SB / 64][MB], fb[SB / 64][NP][NB];
#pragma unroll
    for (int sub = 0; sub < SB / 64; ++sub) {
#pragma unroll
      for (int i = 0; i < MB; ++i) fa[sub][i] = PA::frag(base, lba, wm * (BM / 2) + 16 * i, sub);
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int j = 0; j < NB; ++j)
          fb[sub][p][j] = PB::frag(base + PA::BYTES + p * PB::BYTES, lbb, wn * (BP / 2) + 16 * j, sub);
    }
    issue();   // while the fragments are on their way
#pragma unroll
    for (int sub = 0; sub < SB / 64; ++sub)
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
          for (int j = 0; j < NB; ++j) acc[p][i][j] = T::mfma(fb[sub][p][j], fa[sub][i], acc[p][i][j]);
  }
  __shared__ float s_row[row_scaled(EPI) ? BM : 1];
  if constexpr (row_scaled(EPI))
    if (threadIdx.x < BM) s_row[threadIdx.x] = row_scale<EPI>(g, it.z, m0 + threadIdx.x);
  wait_barrier<0>();   // every wave's copies and reads are done: LDS is free
  // lane: row lane % 16 of its block, columns 4 (lane / 16) .. + 3
  constexpr int COLS = NP * BP / 2;
  const uint32_t turn = lds0 + wid * (BM / 2 * COLS * 4);
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int j = 0; j < NB; ++j)
        turn_in<COLS>(turn, 16 * i + (lane & 15), 4 * (p * NB + j) + (lane >> 4), acc[p][i][j]);
  turn_out<A, EPI, COLS>(g, it.z, int64_t(it.ks) * g.batches + it.z, turn, lane, BM / 2, m0 + wm * (BM / 2),
                         n0 + wn * (BP / 2), s_row + wm * (BM / 2));
}

// ---------------------------------------------------------------- large tile kernel
// 256 x 256 per workgroup of 8 waves (2 x 4, 128 x 64 each), K steps of 64 bytes in a ring of
// four (128 KB).  A step is 32 MFMAs per wave and needs 12 fragments: step s + 3 is copied
// while step s is read, into the slot whose last read ended the step before; a wave waits
// only for its copies of two steps ago (8 of 1 KB stay in flight).
// Waves 4..7 (the other wave of each SIMD) run half a step behind waves 0..3: while one wave
// of a SIMD reads LDS and issues copies, the other feeds the matrix core.
template <Act A, bool AMC, bool BMC, int EPI>
__global__ void __launch_bounds__(512, 1) k_dense_big(DenseArgs g, int mtiles, int ntiles) {
  typedef Num<A> T;
  typedef typename T::acc_t acc_t;
  constexpr bool DUAL = EPI == EPI_SWIGLU;
  constexpr int SEGS = segments(AMC, BMC);
  constexpr int SB = 64;
  constexpr int STEP = SB / T::ESZ;
  constexpr int BP = DUAL ? 128 : 256;              // rows of a B panel
  typedef Panel<A, AMC, 256, SB> PA;
  typedef Panel<A, BMC, BP, SB> PB;
  constexpr int SLOT = 2 * PA::BYTES;               // 16 KB of A, 16 KB of B
  constexpr int MB = 8, NB = 4;                     // 16-blocks per wave
  __shared__ __align__(16) uint8_t ring[4 * SLOT];

  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  const int wm = wid >> 2, wn = wid & 3;
  const Item it = item_of(blockIdx.x, gridDim.x, g.batches, mtiles, ntiles);
  const int m0 = it.mt * 256, n0 = it.nt * BP;
  const int seg_steps = (g.K + STEP - 1) / STEP;
  const int all = seg_steps * SEGS;
  const int per = (all + g.ksplit - 1) / g.ksplit;
  const int s_begin = it.ks * per, s_end = min(all, s_begin + per);
  const uint32_t lds0 = lds_addr(ring);

  // Each wave copies 2 KB of each operand per step (swiglu: waves 0..3 of the gate panel,
  // 4..7 of the up panel).  Past the last step the descriptor is empty: the copy counts, and
  // writes zeros that nothing reads.
  const int cb = DUAL ? 2 * wn : 2 * wid;           // first copy of the wave in its B panel
  int si = s_begin, k_left = 0;                     // the next step to copy, its bytes of K
  typename PA::Feed fda;
  typename PB::Feed fdb;
  auto start = [&](int seg, int step) {
    fda = PA::feed((SEGS == 2 ? seg : it.z) ? g.a[1] : g.a[0], g.lda, g.M, g.K, m0, step);
    fdb = PB::feed((DUAL ? wm : seg) ? g.b[1] : g.b[0], g.ldb, g.N, g.K, n0, step);
    k_left = g.K * T::ESZ - step * SB;
  };
  if (SEGS == 1 || s_begin < seg_steps) start(0, s_begin);
  else start(1, s_begin - seg_steps);
  auto issue = [&]() {
    if constexpr (SEGS == 2)
      if (si == seg_steps) start(1, 0);
    const bool in = si < s_end;
    const uint32_t at = lds0 + uint32_t(si & 3) * SLOT;
    copies<PA, 2>(fda.rsrc(in), at, 2 * wid, lane, g.lda, AMC ? g.M - m0 : k_left);
    copies<PB, 2>(fdb.rsrc(in), at + PA::BYTES + (DUAL ? wm * PB::BYTES : 0), cb, lane, g.ldb, BMC ? g.N - n0 : k_left);
    fda.next();
    fdb.next();
    k_left -= SB;
    ++si;
  };
  const uint32_t lba = PA::lane_base(lane), lbb = PB::lane_base(lane);

  acc_t acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = acc_t{0, 0, 0, 0};
  auto fence = [] { __builtin_amdgcn_sched_barrier(0); };

  issue();
  issue();
  issue();
  asm volatile("s_waitcnt vmcnt(8)\n\ts_barrier" ::: "memory");
  if (wid >= 4) asm volatile("s_barrier" ::: "memory");
  for (int s = s_begin; s < s_end; ++s) {
    const uint32_t p = lds0 + uint32_t(s & 3) * SLOT;
    u32x4_t va[MB], vb[NB];
    // swiglu: blocks 0, 1 of the wave in the gate panel, 2, 3 in the up panel
#pragma unroll
    for (int j = 0; j < NB; ++j)
      vb[j] = DUAL ? PB::frag(p + PA::BYTES + (j / 2) * PB::BYTES, lbb, wn * 32 + 16 * (j % 2), 0)
                   : PB::frag(p + PA::BYTES, lbb, wn * 64 + 16 * j, 0);
#pragma unroll
    for (int i = 0; i < MB; ++i) va[i] = PA::frag(p, lba, wm * 128 + 16 * i, 0);
    issue();   // step s + 3
    // fragments in registers, copies of step s + 1 in LDS
    fence();
    asm volatile("s_waitcnt vmcnt(8) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    fence();
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = T::mfma(vb[j], va[i], acc[i][j]);
    __builtin_amdgcn_s_setprio(0);
    fence();
    asm volatile("s_barrier" ::: "memory");
    fence();
  }
  if (wid < 4) asm volatile("s_barrier" ::: "memory");
  __shared__ float s_row[row_scaled(EPI) ? 256 : 1];
  if constexpr (row_scaled(EPI))
    if (threadIdx.x < 256) s_row[threadIdx.x] = row_scale<EPI>(g, it.z, m0 + threadIdx.x);
  wait_barrier<0>();   // every wave's copies and reads are done: LDS is free
  // lane: row lane % 16 of its block, columns 4 (lane / 16) .. + 3; 64 rows at a time
  const uint32_t turn = lds0 + wid * (64 * 64 * 4);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int i = 0; i < MB / 2; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
        turn_in<64>(turn, 16 * i + (lane & 15), 4 * j + (lane >> 4), acc[h * (MB / 2) + i][j]);
    turn_out<A, EPI, 64>(g, it.z, int64_t(it.ks) * g.batches + it.z, turn, lane, 64, m0 + wm * 128 + h * 64,
                         n0 + wn * (DUAL ? 32 : 64), s_row + wm * 128 + h * 64);
  }
}

// Adds the K slices of a split product in slice order and finishes four columns per thread.
template <Act A, int EPI>
__global__ void __launch_bounds__(256) k_dense_join(DenseArgs g) {
  typedef typename Num<A>::acc_t acc_t;
  typedef typename std::conditional<A == Act::I8, int32_t, float>::type S;
  constexpr int NP = EPI == EPI_SWIGLU ? 2 : 1;
  const uint32_t quads = (g.N + 3) / 4, i = blockIdx.x * 256 + threadIdx.x;   // (plan_us: below 2^32)
  const uint32_t zm = i / quads;
  if (zm >= uint32_t(g.batches) * g.M) return;
  const int n = int(i - zm * quads) * 4;
  const int z = zm >= uint32_t(g.M), m = int(zm) - z * g.M;   // (one batch or two)
  const int count = g.N - n < 4 ? g.N - n : 4;
  const bool vec = count == 4 && (g.N & 3) == 0;
  acc_t v[2];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    v[p] = acc_t{0, 0, 0, 0};
    for (int s = 0; s < g.ksplit; ++s) {
      const S* q = static_cast<const S*>(g.part) + (((int64_t(s) * g.batches + z) * NP + p) * g.M + m) * g.N + n;
      if (vec) {
        v[p] += *reinterpret_cast<const acc_t*>(q);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e < count) v[p][e] += q[e];
      }
    }
  }
  finish4<A, EPI>(g, z, m, n, v[0], v[NP - 1], row_scale<EPI>(g, z, m), col_scales<EPI>(g, n));
}

// ---------------------------------------------------------------- few rows
// Up to 16 rows: bound by reading the weights once.  A wave's fragment is 16 weight rows (16
// columns of y; for swiglu 8 gate and 8 up rows, so that twice as many workgroups share the
// reading); the 8 waves of a workgroup own NF fragments' rows, take the 128-byte K steps in
// turn and feed the matrix core straight from global memory (16 bytes per lane, two loads
// cover a step's whole lines), four steps per turn of the loop, then add their sums through LDS
// in wave order.  The compiler spreads a turn's 16 loads (24 of NF = 2) over its products: 8 (6)
// are in flight at a time, in 64 registers.  2048 / 8192 gated projection, one row: 12.2 us, 5.5
// TB/s (with non-temporal weight loads the second load of a line misses again: 14.6 against
// 14.0 us on another card).
template <Act A, int EPI, int W, int NF>
__global__ void __launch_bounds__(64 * W) k_dense_rows(DenseArgs g) {
  typedef Num<A> T;
  typedef typename T::acc_t acc_t;
  constexpr bool DUAL = EPI == EPI_SWIGLU;
  __shared__ acc_t sums[W][NF][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int row = lane & 15, quarter = (lane >> 4) * 16;
  constexpr int COLS = DUAL ? 8 : 16;   // columns per fragment
  const int n0 = blockIdx.x * (COLS * NF);
  const int64_t kb = int64_t(g.K) * T::ESZ;   // bytes of a row (a multiple of 16)
  const void* wb = DUAL && row >= 8 ? g.b[1] : g.b[0];
  const uint8_t* wp[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f)
    wp[f] = static_cast<const uint8_t*>(wb) + min(n0 + f * COLS + (DUAL ? row & 7 : row), g.N - 1) * kb + quarter;
  const uint8_t* xp = static_cast<const uint8_t*>(g.a[0]) + min(row, g.M - 1) * kb + quarter;
  acc_t acc[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) acc[f] = acc_t{0, 0, 0, 0};

  const int full = int(kb / kStepBytes);
  int s = wave;
  auto steps = [&](auto u_c) {
    constexpr int N = decltype(u_c)::value;
    u32x4_t w[N][2][NF], x[N][2];
#pragma unroll
    for (int u = 0; u < N; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t at = int64_t(s + u * W) * kStepBytes + h * 64;
#pragma unroll
        for (int f = 0; f < NF; ++f)
          w[u][h][f] = *reinterpret_cast<const u32x4_t*>(wp[f] + at);
        x[u][h] = *reinterpret_cast<const u32x4_t*>(xp + at);
      }
#pragma unroll
    for (int u = 0; u < N; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int f = 0; f < NF; ++f) acc[f] = T::mfma(w[u][h][f], x[u][h], acc[f]);
    s += N * W;
  };
  while (s + 3 * W < full) steps(std::integral_constant<int, 4>{});
  if (s + W < full) steps(std::integral_constant<int, 2>{});
  if (s < full) steps(std::integral_constant<int, 1>{});
  if (s == full && kb % kStepBytes) {   // the K tail: lanes past the row's end hold zeros
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t at = int64_t(full) * kStepBytes + h * 64;
      const bool in = at + quarter < kb;
      const u32x4_t x = in ? *reinterpret_cast<const u32x4_t*>(xp + at) : u32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int f = 0; f < NF; ++f)
        acc[f] = T::mfma(in ? *reinterpret_cast<const u32x4_t*>(wp[f] + at) : u32x4_t{0, 0, 0, 0}, x, acc[f]);
    }
  }
#pragma unroll
  for (int f = 0; f < NF; ++f) sums[wave][f][lane] = acc[f];
  __syncthreads();
  if (wave >= NF) return;
  acc_t v = sums[0][wave][lane];
#pragma unroll
  for (int w = 1; w < W; ++w) v += sums[w][wave][lane];
  const int m = row, n = n0 + wave * COLS + 4 * (lane >> 4);
  if constexpr (DUAL) {   // quarters 0, 1: gate columns; 2, 3: the same columns' up values
    acc_t up;
#pragma unroll
    for (int i = 0; i < 4; ++i) up[i] = __shfl_xor(v[i], 32, 64);
    if (lane < 32) finish4<A, EPI>(g, 0, m, n, v, up, 0.f, col_scales<EPI>(g, n));
  } else {
    finish4<A, EPI>(g, 0, m, n, v, v, row_scale<EPI>(g, 0, m), col_scales<EPI>(g, n));
  }
}

// ---------------------------------------------------------------- element-wise kernels
// dg and du of 8 elements, columns c .. c + 7 of a token's row.
template <bool F16>
Q4_DEVICE void swiglu_grad8(const uint16_t* __restrict__ dh, const float* __restrict__ gu, int64_t row, int64_t inter,
                            int64_t c, float a[8], float b[8]) {
  f32x4_t g[2], u[2];
  uint16_t d[8];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    g[j] = __builtin_nontemporal_load(reinterpret_cast<const f32x4_t*>(gu + row * 2 * inter + c + 4 * j));
    u[j] = __builtin_nontemporal_load(reinterpret_cast<const f32x4_t*>(gu + row * 2 * inter + inter + c + 4 * j));
  }
  *reinterpret_cast<uint4*>(d) = load16_stream(dh + row * inter + c);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float gv = g[e / 4][e % 4], uv = u[e / 4][e % 4];
    const float dv = F16 ? f16_bits_to_f32(d[e]) : bf16_to_f32(d[e]);
    const float sig = __builtin_amdgcn_rcpf(1.0f + __expf(-gv));
    a[e] = dv * uv * sig * (1.0f + gv * (1.0f - sig));
    b[e] = dv * gv * sig;
  }
}

// dg and du in bf16: bound by memory (g, u in fp32 and dh in, dg and du out: 14 bytes per
// element).  g and u are kept in fp32: rounding them to 16 bits as well made the bf16
// gradients 1.8 times as far from the 64-bit ones as one rounding of the result does, fp32
// 1.4 times.  The rest is the rounding of dg and du themselves: as matrix-core operands they
// have the type of x and the weights.  With a second operand for what that rounding leaves the
// gradients are as near as one rounding (0.0017 instead of 0.0023 relative), but all three
// products double: 524 -> 981 us backward at 4096 x 2048 x 8192.
__global__ void __launch_bounds__(256) k_swiglu_grad(const uint16_t* __restrict__ dh, const float* __restrict__ gu,
                                                     int64_t t, int64_t inter, uint16_t* __restrict__ dg,
                                                     uint16_t* __restrict__ du) {
  const int64_t vecs = inter / 8;
  const int64_t step = int64_t(gridDim.x) * 256;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < t * vecs; i += step) {
    const int64_t row = i / vecs, c = (i - row * vecs) * 8;
    float va[8], vb[8];
    swiglu_grad8<false>(dh, gu, row, inter, c, va, vb);
    uint16_t a[8], b[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] = to16(va[e], 2), b[e] = to16(vb[e], 2);
    *reinterpret_cast<uint4*>(dg + row * inter + c) = *reinterpret_cast<const uint4*>(a);
    *reinterpret_cast<uint4*>(du + row * inter + c) = *reinterpret_cast<const uint4*>(b);
  }
}

// dg and du in fp16.  The type holds 2^-24 to 2^16 and the fp32 values can lie outside it where
// the gradients do not (dh of 2^12 and u of 2^8, times weights of 2^-12), so each operand takes
// powers of two along the axis that the product keeps: dx keeps the tokens, dw the columns.
//   dx  = 2^r_t (2^-r_t dg Wg + 2^-r_t du Wu),   dWg = 2^c_i ((2^-c_i dg)^T x),  dWu likewise
// which takes the largest finite magnitude of each row and column first, a pass of its own over
// g, u and dh (10 bytes per element), and two sets of operands (8 bytes written, not 4): the
// backward pass of 4096 x 2048 x 8192 takes 657 us, unscaled 555, of 777 x 1000 x 2728 71 and 56.
// Scaled, that magnitude lies in [2^14, 2^15): nothing overflows, and an element loses bits
// only below 2^-28 of it.
constexpr int kMaxGroup = 512;   // columns of a wave's row maximum

// Rows per partial column maximum: 8 (of 32, 777 x 1000 x 2728 has 150 workgroups and takes 74 us),
// more where that made over 2048 workgroups.
int64_t grad_rows(int64_t t, int64_t inter) {
  const int64_t groups = (inter + kMaxGroup - 1) / kMaxGroup;
  const int64_t chunks = std::max<int64_t>(1, 2048 / groups);
  return std::max<int64_t>(8, (t + chunks - 1) / chunks);
}

// rmax [t][groups]: of a token's dg and du over 512 columns; cmax [chunks][2][inter]: of dg and
// of du over the chunk's rows.
__global__ void __launch_bounds__(256) k_swiglu_grad_max(const uint16_t* __restrict__ dh, const float* __restrict__ gu,
                                                         int64_t t, int64_t inter, int64_t rows, uint32_t groups,
                                                         float* __restrict__ rmax, float* __restrict__ cmax) {
  __shared__ float s[4][2][kMaxGroup];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t group = blockIdx.x % groups, chunk = blockIdx.x / groups;
  const int64_t c = int64_t(group) * kMaxGroup + lane * 8;
  const int64_t end = int64_t(chunk + 1) * rows < t ? int64_t(chunk + 1) * rows : t;
  float ca[8], cb[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) ca[e] = cb[e] = 0.f;
  for (int64_t row = int64_t(chunk) * rows + wave; row < end; row += 4) {
    float m = 0.f;
    if (c < inter) {
      float a[8], b[8];
      swiglu_grad8<true>(dh, gu, row, inter, c, a, b);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // (infinities and NaN stay what they are at any scale)
        const float fa = fabsf(a[e]) < __builtin_inff() ? fabsf(a[e]) : 0.f;
        const float fb = fabsf(b[e]) < __builtin_inff() ? fabsf(b[e]) : 0.f;
        ca[e] = fmaxf(ca[e], fa), cb[e] = fmaxf(cb[e], fb);
        m = fmaxf(m, fmaxf(fa, fb));
      }
    }
    m = wave_max(m);
    if (lane == 0) rmax[row * groups + group] = m;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) s[wave][0][lane * 8 + e] = ca[e], s[wave][1][lane * 8 + e] = cb[e];
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * kMaxGroup; i += 256) {
    const int p = i / kMaxGroup, k = i % kMaxGroup;
    const int64_t col = int64_t(group) * kMaxGroup + k;
    if (col < inter)
      cmax[(int64_t(chunk) * 2 + p) * inter + col] = fmaxf(fmaxf(s[0][p][k], s[1][p][k]), fmaxf(s[2][p][k], s[3][p][k]));
  }
}

// The power of two s with m / s in [2^14, 2^15), within [2^-100, 2^113]: what is smaller than
// 2^-86 to begin with vanishes in any fp16 gradient.
Q4_DEVICE float pow2_scale(float m) {
  const int e = int(__float_as_uint(m) >> 23) - 127 - 14;
  return m > 0.f ? __uint_as_float(uint32_t(max(e, -100) + 127) << 23) : 1.f;
}
// 1 / s of a power of two.
Q4_DEVICE float pow2_inverse(float s) { return __uint_as_float((254u << 23) - __float_as_uint(s)); }

// Scales from the maxima: cscale [2][inter] (workgroups of 64 columns by 16 waves, which take
// every 16th chunk), then rscale [t] (a wave per token).
__global__ void __launch_bounds__(1024) k_swiglu_grad_scales(const float* __restrict__ rmax,
                                                             const float* __restrict__ cmax, int64_t t, int64_t inter,
                                                             int chunks, uint32_t groups, uint32_t col_wgs,
                                                             float* __restrict__ rscale, float* __restrict__ cscale) {
  __shared__ float s[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float m = 0.f;
  if (blockIdx.x < col_wgs) {
    const int64_t c = int64_t(blockIdx.x) * 64 + lane;
    if (c < 2 * inter)
#pragma unroll 4
      for (int k = wave; k < chunks; k += 16) m = fmaxf(m, cmax[int64_t(k) * 2 * inter + c]);
    s[wave][lane] = m;
    __syncthreads();
    if (wave != 0 || c >= 2 * inter) return;
#pragma unroll
    for (int w = 1; w < 16; ++w) m = fmaxf(m, s[w][lane]);
    cscale[c] = pow2_scale(m);
  } else {
    const int64_t row = int64_t(blockIdx.x - col_wgs) * 16 + wave;
    if (row >= t) return;
    for (uint32_t k = lane; k < groups; k += 64) m = fmaxf(m, rmax[row * groups + k]);
    m = wave_max(m);
    if (lane == 0) rscale[row] = pow2_scale(m);
  }
}

// dg and du scaled by row (row_g, row_u: dx) and by column (col_g, col_u: dw).
__global__ void __launch_bounds__(256) k_swiglu_grad_scaled(const uint16_t* __restrict__ dh,
                                                            const float* __restrict__ gu, int64_t t, int64_t inter,
                                                            const float* __restrict__ rscale,
                                                            const float* __restrict__ cscale,
                                                            uint16_t* __restrict__ row_g, uint16_t* __restrict__ row_u,
                                                            uint16_t* __restrict__ col_g,
                                                            uint16_t* __restrict__ col_u) {
  const int64_t vecs = inter / 8;
  const int64_t step = int64_t(gridDim.x) * 256;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < t * vecs; i += step) {
    const int64_t row = i / vecs, c = (i - row * vecs) * 8;
    float va[8], vb[8];
    swiglu_grad8<true>(dh, gu, row, inter, c, va, vb);
    const float r = pow2_inverse(rscale[row]);
    uint16_t a[8], b[8], ca[8], cb[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      a[e] = to16(va[e] * r, 1), b[e] = to16(vb[e] * r, 1);
      ca[e] = to16(va[e] * pow2_inverse(cscale[c + e]), 1);
      cb[e] = to16(vb[e] * pow2_inverse(cscale[inter + c + e]), 1);
    }
    *reinterpret_cast<uint4*>(row_g + row * inter + c) = *reinterpret_cast<const uint4*>(a);
    *reinterpret_cast<uint4*>(row_u + row * inter + c) = *reinterpret_cast<const uint4*>(b);
    *reinterpret_cast<uint4*>(col_g + row * inter + c) = *reinterpret_cast<const uint4*>(ca);
    *reinterpret_cast<uint4*>(col_u + row * inter + c) = *reinterpret_cast<const uint4*>(cb);
  }
}

// One workgroup per weight row: amax, then the codes.
template <int DT>
__global__ void __launch_bounds__(256) k_quantize8_rows(const void* __restrict__ w, int64_t k, int8_t* __restrict__ q,
                                                        float* __restrict__ s, int32_t* flags) {
  __shared__ float red[4];
  const int64_t row = blockIdx.x;
  auto get = [&](int64_t i) -> float {
    if constexpr (DT == 0) return static_cast<const float*>(w)[row * k + i];
    else if constexpr (DT == 1) return f16_bits_to_f32(static_cast<const uint16_t*>(w)[row * k + i]);
    else return bf16_to_f32(static_cast<const uint16_t*>(w)[row * k + i]);
  };
  float mx = 0.f;
  bool bad = false;
  for (int64_t i = threadIdx.x; i < k; i += 256) {
    const float v = get(i);
    bad |= !(fabsf(v) < __builtin_inff());
    mx = fmaxf(mx, fabsf(v));
  }
  if (bad && flags) atomicOr(flags, 1);
  mx = wave_max(mx);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = mx;
  __syncthreads();
  mx = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  const float sc = mx / 127.0f;
  for (int64_t i = threadIdx.x; i < k; i += 256)
    q[row * k + i] = sc > 0.f ? int8_t(int(fminf(fmaxf(rintf(get(i) / sc), -127.f), 127.f))) : int8_t(0);
  if (threadIdx.x == 0) s[row] = sc;
}

// ---------------------------------------------------------------- launches
int64_t part_bytes(const Plan& p, int64_t m, int64_t n, int panels, int batches) {
  return p.ksplit > 1 ? int64_t(p.ksplit) * batches * panels * m * n * 4 : 0;
}

template <Act A, bool AMC, bool BMC, int EPI>
hipError_t launch_tiles(DenseArgs g, const Plan& p, hipStream_t st) {
  constexpr int NP = EPI == EPI_SWIGLU ? 2 : 1;
  g.ksplit = p.ksplit;
  const int mt = int(ceil_div(g.M, p.tile)), nt = int(ceil_div(int64_t(g.N) * NP, p.tile));
  const unsigned grid = unsigned(int64_t(mt) * nt * g.batches * p.ksplit);
  if (p.tile == 256)
    hipLaunchKernelGGL((k_dense_big<A, AMC, BMC, EPI>), dim3(grid), dim3(512), 0, st, g, mt, nt);
  else if (p.tile == 128)
    hipLaunchKernelGGL((k_dense<A, AMC, BMC, 128, 128, 64, 4, EPI>), dim3(grid), dim3(256), 0, st, g, mt, nt);
  else
    hipLaunchKernelGGL((k_dense<A, AMC, BMC, 64, 64, 128, 3, EPI>), dim3(grid), dim3(256), 0, st, g, mt, nt);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.ksplit == 1) return e;
  const int64_t threads = int64_t(g.batches) * g.M * ((g.N + 3) / 4);
  hipLaunchKernelGGL((k_dense_join<A, EPI>), dim3(unsigned(ceil_div(threads, 256))), dim3(256), 0, st, g);
  return hipGetLastError();
}

template <Act A, int EPI, int W, int NF>
hipError_t launch_rows_as(const DenseArgs& g, hipStream_t st) {
  const dim3 grid(unsigned(ceil_div(g.N, (EPI == EPI_SWIGLU ? 8 : 16) * NF)));
  hipLaunchKernelGGL((k_dense_rows<A, EPI, W, NF>), grid, dim3(64 * W), 0, st, g);
  return hipGetLastError();
}

// Two fragments per wave halve the reads of x, which count from a few rows on, as long as
// enough workgroups are left: 7168 x 7168 INT8 12.4 -> 11.1 us at 5 rows, 15.1 -> 12.3 at 16,
// gated 2048 / 8192 13.4 -> 12.3 at 5; but INT8 8192 x 2048, 64 workgroups instead of 128, 9.6
// -> 13.0 at 16, gated 7168 / 2048 15.1 -> 21.2.  (Where the rule takes two and K is long, a
// gated projection can lose: 4096 / 6144 20.5 -> 23.0 at 5 rows, 24.9 -> 25.1 at 16.)
template <Act A, int EPI>
hipError_t launch_rows(const DenseArgs& g, hipStream_t st) {
  const int64_t wgs = ceil_div(g.N, EPI == EPI_SWIGLU ? 16 : 32);
  return g.M > 4 && wgs >= 192 ? launch_rows_as<A, EPI, 8, 2>(g, st) : launch_rows_as<A, EPI, 8, 1>(g, st);
}

}  // namespace

hipError_t launch_quantize8_rows(const void* w, int dtype, int64_t n, int64_t k, int8_t* q, float* s, int32_t* flags,
                                 hipStream_t st) {
  const dim3 grid{unsigned(n)}, block(256);
  if (dtype == 0) hipLaunchKernelGGL(k_quantize8_rows<0>, grid, block, 0, st, w, k, q, s, flags);
  else if (dtype == 1) hipLaunchKernelGGL(k_quantize8_rows<1>, grid, block, 0, st, w, k, q, s, flags);
  else hipLaunchKernelGGL(k_quantize8_rows<2>, grid, block, 0, st, w, k, q, s, flags);
  return hipGetLastError();
}

int64_t int8_linear_workspace(int64_t t, int64_t k, int64_t n) {
  return t == 0 ? 0 : part_bytes(int8_plan(t, k, n), t, n, 1, 1);
}

hipError_t launch_int8_linear(const int8_t* q, const float* s, int64_t t, int64_t k, const int8_t* wq, const float* ws,
                              int64_t n, const float* bias, int y_dtype, void* y, void* work, hipStream_t st) {
  DenseArgs g{};
  g.a[0] = g.a[1] = q;
  g.b[0] = g.b[1] = wq;
  g.lda = g.ldb = k;
  g.M = int32_t(t), g.N = int32_t(n), g.K = int32_t(k);
  g.batches = g.ksplit = 1;
  g.c[0] = y;
  g.ldc = n;
  g.c_dtype = y_dtype;
  g.s_row = s;
  g.s_col = ws;
  g.bias = bias;
  g.part = work;
  const Plan p = int8_plan(t, k, n);
  return p.tile == 0 ? launch_rows<Act::I8, EPI_INT8>(g, st) : launch_tiles<Act::I8, false, false, EPI_INT8>(g, p, st);
}

int64_t swiglu_linear_workspace(int64_t t, int64_t h, int64_t i) {
  return t == 0 ? 0 : part_bytes(swiglu_plan(t, h, i), t, i, 2, 1);
}

hipError_t launch_swiglu_linear(const void* x, const void* wg, const void* wu, int64_t t, int64_t h, int64_t i, int f16,
                                void* out, float* gu, void* work, hipStream_t st) {
  DenseArgs g{};
  g.a[0] = g.a[1] = x;
  g.b[0] = wg, g.b[1] = wu;
  g.lda = g.ldb = h;
  g.M = int32_t(t), g.N = int32_t(i), g.K = int32_t(h);
  g.batches = g.ksplit = 1;
  g.c[0] = out;
  g.ldc = i;
  g.c_dtype = f16 ? 1 : 2;
  g.gu = gu;
  g.part = work;
  const Plan p = swiglu_plan(t, h, i);
  if (p.tile == 0)
    return f16 ? launch_rows<Act::F16, EPI_SWIGLU>(g, st) : launch_rows<Act::BF16, EPI_SWIGLU>(g, st);
  return f16 ? launch_tiles<Act::F16, false, false, EPI_SWIGLU>(g, p, st)
             : launch_tiles<Act::BF16, false, false, EPI_SWIGLU>(g, p, st);
}

// Workspace of the gradients: the K slices of whichever product splits K, dg and du [t][i]
// (in fp16 scaled by row, and once more scaled by column, with the scales and the maxima that
// they come from).  One size for both types.
struct GradWork {
  Plan dx, dw;
  void* part;
  uint16_t *g, *u, *col_g, *col_u;
  float *rscale, *cscale, *rmax, *cmax;
  int64_t bytes;
};
GradWork grad_work(void* base, int64_t t, int64_t h, int64_t i) {
  const int64_t groups = ceil_div(i, kMaxGroup);
  GradWork w{};
  w.dx = dx_plan(t, h, i);
  w.dw = dw_plan(t, h, i);
  auto take = [&](int64_t bytes) {
    uint8_t* p = static_cast<uint8_t*>(base) + w.bytes;
    w.bytes += align256(bytes);
    return static_cast<void*>(p);
  };
  auto half = [&] { return static_cast<uint16_t*>(take(t * i * 2)); };
  auto floats = [&](int64_t n) { return static_cast<float*>(take(n * 4)); };
  w.part = take(std::max(part_bytes(w.dx, t, h, 1, 1), part_bytes(w.dw, i, h, 1, 2)));
  w.g = half(), w.u = half(), w.col_g = half(), w.col_u = half();
  w.rscale = floats(t), w.cscale = floats(2 * i);
  w.rmax = floats(t * groups), w.cmax = floats(ceil_div(t, grad_rows(t, i)) * 2 * i);
  return w;
}
int64_t swiglu_linear_bwd_workspace(int64_t t, int64_t h, int64_t i) {
  return t == 0 ? 0 : grad_work(nullptr, t, h, i).bytes;
}

hipError_t launch_swiglu_linear_bwd(const void* dh, const void* x, const void* wg, const void* wu, const float* gu,
                                    int64_t t, int64_t h, int64_t i, int f16, void* dx, void* dwg, void* dwu,
                                    void* work, hipStream_t st) {
  const GradWork w = grad_work(work, t, h, i);
  if (t > 0) {
    const unsigned grid = unsigned(std::min<int64_t>(ceil_div(t * (i / 8), 256), 4096));
    const auto* d = static_cast<const uint16_t*>(dh);
    if (f16) {
      const int64_t rows = grad_rows(t, i), chunks = ceil_div(t, rows);
      const unsigned groups = unsigned(ceil_div(i, kMaxGroup)), col_wgs = unsigned(ceil_div(2 * i, 64));
      hipLaunchKernelGGL(k_swiglu_grad_max, dim3(unsigned(groups * chunks)), dim3(256), 0, st, d, gu, t, i, rows, groups,
                         w.rmax, w.cmax);
      hipLaunchKernelGGL(k_swiglu_grad_scales, dim3(unsigned(col_wgs + ceil_div(t, 16))), dim3(1024), 0, st, w.rmax,
                         w.cmax, t, i, int(chunks), groups, col_wgs, w.rscale, w.cscale);
      hipLaunchKernelGGL(k_swiglu_grad_scaled, dim3(grid), dim3(256), 0, st, d, gu, t, i, w.rscale, w.cscale, w.g, w.u,
                         w.col_g, w.col_u);
    } else {
      hipLaunchKernelGGL(k_swiglu_grad, dim3(grid), dim3(256), 0, st, d, gu, t, i, w.g, w.u);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  DenseArgs g{};
  g.c_dtype = f16 ? 1 : 2;
  g.ksplit = 1;
  g.part = w.part;
  g.ldc = h;
  g.N = int32_t(h);
  if (t > 0) {   // dx = dg Wg + du Wu: K runs over the gate rows, then the up rows
    g.a[0] = w.g, g.a[1] = w.u;
    g.b[0] = wg, g.b[1] = wu;
    g.lda = i, g.ldb = h;
    g.M = int32_t(t), g.K = int32_t(i);
    g.batches = 1;
    g.c[0] = g.c[1] = dx;
    g.s_row = w.rscale;
    const hipError_t e = f16 ? launch_tiles<Act::F16, false, true, EPI_SCALED>(g, w.dx, st)
                             : launch_tiles<Act::BF16, false, true, EPI_STORE>(g, w.dx, st);
    if (e != hipSuccess) return e;
  }
  // dWg = dg^T x and dWu = du^T x as two batches (t == 0: no K step, zeros)
  g.a[0] = f16 ? w.col_g : w.g, g.a[1] = f16 ? w.col_u : w.u;
  g.b[0] = g.b[1] = x;
  g.lda = i, g.ldb = h;
  g.M = int32_t(i), g.K = int32_t(t);
  g.batches = 2;
  g.c[0] = dwg, g.c[1] = dwu;
  g.s_row = w.cscale;
  return f16 && t > 0 ? launch_tiles<Act::F16, true, true, EPI_SCALED>(g, w.dw, st)
                      : launch_tiles<Act::BF16, true, true, EPI_STORE>(g, w.dw, st);
}

}  // namespace q4
