// Tokens sorted by expert and back, with their weights, and the gradients of both.
//
//   dispatch   xp[pos(t, j)] = x[t]                      pos: slots t k + j in order of (expert, slot)
//   back       dx[t] = sum_j dxp[pos(t, j)]              (combine without weights)
//   combine    out[t] = sum_j w[t][j] y[pos(t, j)] (+ add[t])
//   back       dy[pos(t, j)] = w[t][j] dout[t],  dw[t][j] = <dout[t], y[pos(t, j)]>
//
// All are bound by the rows' bytes.  Sums are fp32 in ascending j, so equal inputs give equal
// bits; nothing is added by atomics.
#include <algorithm>
#include <type_traits>

#include "e4m3.h"
#include "tokens.h"
#include "tokens_plan.h"

namespace q4 {

namespace {

constexpr int kThreads = 256;
constexpr int64_t kCacheBytes = int64_t(256) << 20;   // the last-level cache

// Slots that a workgroup ranks against each other: a range of whole tokens of at most this many
// slots (one token where it has more).
constexpr int kRangeSlots = 1024;
// Up to this many slots there is one range, and each workgroup finds the positions by itself: one
// launch instead of three (a call of 500 tokens of 2048, k = 4: 12.8 us against 20.2; 500 of 7168,
// k = 8, 4000 slots: 26.3 against 21.7).
constexpr int64_t kOneRange = 2048;

int64_t range_tokens(int64_t t, int32_t k) {
  return t * k <= kOneRange ? std::max<int64_t>(1, t) : std::max<int64_t>(1, kRangeSlots / k);
}
int64_t ranges(int64_t t, int32_t k) {
  const int64_t r = range_tokens(t, k);
  return (t + r - 1) / r;
}

// Expert of a slot, e for one that is not held.
Q4_DEVICE int slot_local(const int32_t* ids, int64_t s, int first, int e) {
  const uint32_t x = uint32_t(ids[s]) - uint32_t(first);
  return x < uint32_t(e) ? int(x) : e;
}

// use(i, expert of slot s0 + i) for i below n, a workgroup's threads side by side, 8 loads in flight.
template <typename F>
Q4_DEVICE void each_slot(const int32_t* ids, int64_t s0, int n, int first, int e, F use) {
  constexpr int U = 8;
  for (int i0 = threadIdx.x; i0 < n; i0 += U * kThreads) {
    int x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) x[u] = i0 + u * kThreads < n ? slot_local(ids, s0 + i0 + u * kThreads, first, e) : 0;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u * kThreads < n) use(i0 + u * kThreads, x[u]);
  }
}

// In-place exclusive scan of n ints in LDS by 64 * W threads; returns the total.
template <int W>
__device__ int32_t scan_lds(int32_t* v, int n, int32_t* tot) {
  const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
  const int per = (n + 64 * W - 1) / (64 * W);
  const int beg = min(n, tid * per), end = min(n, beg + per);
  int32_t sum = 0;
  for (int i = beg; i < end; ++i) sum += v[i];
  int32_t inc = sum;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int32_t u = __shfl_up(inc, o, 64);
    if (lane >= o) inc += u;
  }
  if (lane == 63) tot[wid] = inc;
  __syncthreads();
  int32_t run = inc - sum, total = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w < wid) run += tot[w];
    total += tot[w];
  }
  for (int i = beg; i < end; ++i) {
    const int32_t x = v[i];
    v[i] = run;
    run += x;
  }
  __syncthreads();
  return total;
}

// Slots per expert (and of none) of each range.
__global__ void __launch_bounds__(kThreads) k_order_count(const int32_t* __restrict__ ids, int64_t t, int32_t k,
                                                          int32_t first, int32_t e, int64_t per,
                                                          int32_t* __restrict__ cnt) {
  extern __shared__ int32_t lds[];   // [e + 1]
  for (int x = threadIdx.x; x <= e; x += kThreads) lds[x] = 0;
  __syncthreads();
  const int64_t beg = int64_t(blockIdx.x) * per * k, end = std::min<int64_t>(t * k, beg + per * k);
  each_slot(ids, beg, int(end - beg), first, e, [&](int, int x) { atomicAdd(&lds[x], 1); });
  __syncthreads();
  for (int x = threadIdx.x; x <= e; x += kThreads) cnt[int64_t(blockIdx.x) * (e + 1) + x] = lds[x];
}

// The ranges' counts [nr][e + 1] become each range's first position per expert; offsets.  Thread
// (part, x) adds a part of the ranges of expert x, as many parts as 1024 threads make.
__global__ void __launch_bounds__(1024) k_order_plan(int32_t* __restrict__ cnt, int nr, int32_t e, int parts,
                                                     int32_t* __restrict__ offsets) {
  extern __shared__ int32_t lds[];   // [e + 1], [parts][e + 1]
  __shared__ int32_t tot[16];
  constexpr int U = 8;   // ranges in flight
  const int64_t ld = e + 1;
  int32_t* sums = lds + e + 1;
  const int per = (nr + parts - 1) / parts;
  auto walk = [&](int x, int r0, int r1, auto use) {
    for (int r = r0; r < r1; r += U) {
      int32_t c[U];
#pragma unroll
      for (int u = 0; u < U; ++u) c[u] = r + u < r1 ? cnt[(r + u) * ld + x] : 0;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (r + u < r1) use(r + u, c[u]);
    }
  };
  for (int i = threadIdx.x; i < parts * (e + 1); i += 1024) {
    const int part = i / (e + 1), x = i - part * (e + 1);
    int32_t run = 0;
    walk(x, part * per, min(nr, (part + 1) * per), [&](int, int32_t c) { run += c; });
    sums[i] = run;
  }
  __syncthreads();
  for (int x = threadIdx.x; x <= e; x += 1024) {
    int32_t run = 0;
    for (int p = 0; p < parts; ++p) {
      const int32_t c = sums[p * (e + 1) + x];
      sums[p * (e + 1) + x] = run;
      run += c;
    }
    lds[x] = run;
  }
  __syncthreads();
  scan_lds<16>(lds, e + 1, tot);
  for (int x = threadIdx.x; x <= e; x += 1024) offsets[x] = lds[x];   // (x == e: the held slots)
  for (int i = threadIdx.x; i < parts * (e + 1); i += 1024) {
    const int part = i / (e + 1), x = i - part * (e + 1);
    int32_t run = lds[x] + sums[i];
    walk(x, part * per, min(nr, (part + 1) * per), [&](int r, int32_t c) {
      cnt[r * ld + x] = run;
      run += c;
    });
  }
}

// Offsets of a call with one range, by the last workgroup of the dispatch.
__device__ void offsets_of(const DispatchArgs& a, int32_t* hist, int32_t* tot) {
  for (int x = threadIdx.x; x <= a.e; x += kThreads) hist[x] = 0;
  __syncthreads();
  each_slot(a.ids, 0, int(a.t * a.k), a.first, a.e, [&](int, int x) { atomicAdd(&hist[x], 1); });
  __syncthreads();
  scan_lds<kThreads / 64>(hist, a.e + 1, tot);
  for (int x = threadIdx.x; x <= a.e; x += kThreads) a.offsets[x] = hist[x];
}

// A workgroup takes TPW consecutive tokens of one range and the columns of block blockIdx.y.
// Positions: a slot's key is (expert, slot); its position is the number of smaller keys, which
// the waves count by ballots over the range's experts in LDS -- all slots with one range, else the
// same expert's slots of the range, on top of the range's first position.  Then the rows go out,
// each token read once and written k times.  NT: rows larger than the last-level cache are written
// past it (4096 tokens of 7168, k = 8: 121 -> 106 us).
//
// 4096 tokens of 7168, k = 8, take 93 us, the rows' bytes.  Where a rank holds an eighth of the slots the ranking
// remains: 39 us as codes, 14 to 18 for the bytes; vector instructions (825 a wave, for the ranks of two
// slots among 1024 and for 1792 codes) take 64 % of the cycles, the waits for slots, ranks and rows in
// turn the rest.  4096 of 2048, k = 2, by waves: 15.5 us against 10 for the bytes, where waves wait for
// these three quarters of their time.
template <bool QUANT, int DT, int TPW, bool NT>
__global__ void __launch_bounds__(kThreads) k_dispatch(DispatchArgs a, int64_t per, const int32_t* __restrict__ base,
                                                       int64_t col_block) {
  typedef Elem<DT> E;
  extern __shared__ int32_t lds[];
  __shared__ int32_t tot[kThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
  const int64_t groups = (per + TPW - 1) / TPW;   // workgroups per range
  const int64_t range = blockIdx.x / groups, tok0 = range * per;
  if (tok0 >= a.t) {   // one range: the workgroup behind the tokens
    if (blockIdx.y == 0) offsets_of(a, lds, tot);
    return;
  }
  const int64_t tokens = std::min<int64_t>(per, a.t - tok0);
  const int64_t mine = (blockIdx.x - range * groups) * TPW;   // first token within the range
  const int nt = int(std::min<int64_t>(TPW, tokens - mine));
  if (nt <= 0) return;
  const int n = int(tokens) * a.k, ns = nt * a.k, s0 = int(mine) * a.k;   // slots of the range, the workgroup's
  int32_t* pos = lds;                                      // [TPW k]
  uint16_t* ex = reinterpret_cast<uint16_t*>(lds + TPW * a.k);   // [slots of a range]
  const int64_t slot0 = tok0 * a.k;
  // the thread's first columns are on their way while the slots are ranked
  constexpr int TPT = kThreads / TPW;   // threads per token
  constexpr int VEC = QUANT ? 8 : E::VEC, RAWS = VEC / E::VEC;
  const int tk = min(tid / TPT, nt - 1), l = tid % TPT;
  const int64_t row = tok0 + mine + tk;
  const int64_t c0 = int64_t(blockIdx.y) * col_block, c1 = std::min<int64_t>(a.h, c0 + col_block);
  typename E::Raw raw[RAWS];
  auto load = [&](int64_t c) {
#pragma unroll
    for (int i = 0; i < RAWS; ++i) raw[i] = E::load(a.x, row * a.h + c + i * E::VEC);
  };
  if (c0 + l * VEC + VEC <= c1) load(c0 + l * VEC);
  each_slot(a.ids, slot0, n, a.first, a.e, [&](int i, int x) { ex[i] = uint16_t(x); });
  __syncthreads();
  // (the experts of U 64 slots stay in registers while the wave's slots are ranked against them)
  constexpr int U = 16;
  for (int i0 = 0; i0 < n; i0 += 64 * U) {
    int x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) x[u] = i0 + 64 * u + lane < n ? int(ex[i0 + 64 * u + lane]) : 0x10000;
    for (int j = wid; j < ns; j += kThreads / 64) {
      const int xj = __builtin_amdgcn_readfirstlane(int(ex[s0 + j]));
      int c = 0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool earlier = i0 + 64 * u + lane < s0 + j;
        c += __popcll(__ballot(base ? x[u] == xj && earlier : x[u] < xj + (earlier ? 1 : 0)));
      }
      if (lane == 0) pos[j] = i0 ? pos[j] + c : c;
    }
  }
  __syncthreads();
  for (int j = tid; j < ns; j += kThreads) {
    const int xj = ex[s0 + j];
    const int32_t p = pos[j] + (base ? base[range * (a.e + 1) + xj] : 0);
    const bool held = xj < a.e;
    pos[j] = held ? p : -1;
    if (blockIdx.y == 0) {
      a.perm[p] = held ? int32_t(slot0 + s0 + j) : -1;
      a.inv[slot0 + s0 + j] = held ? p : -1;
    }
  }
  __syncthreads();
  if (tid / TPT >= nt) return;
  const int32_t* p = pos + tk * a.k;
  if constexpr (QUANT) {
    // 16 lanes hold a group's 128 columns
    const int64_t slots = a.t * a.k;
    for (int64_t c = c0 + l * 8; c < (c1 + 127) / 128 * 128; c += TPT * 8) {
      float v[8], m = 0.f;
      const bool in = c < c1;   // (h is a multiple of 16)
      if (in && c >= c0 + TPT * 8) load(c);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = in ? E::value(raw[i / E::VEC], i % E::VEC) : 0.f;
        m = fmaxf(m, magnitude(v[i]));
      }
      const float s = e4m3_scale(row16_max(m));
      const u32x2_t q = e4m3_codes8(v, s);
      for (int j = 0; j < a.k; ++j) {
        const int32_t at = p[j];
        if (at < 0) continue;
        if (in) *reinterpret_cast<u32x2_t*>(a.q + at * a.h + c) = q;
        if ((l & 15) == 0) a.s[(c >> 7) * slots + at] = s;
      }
    }
  } else {
    for (int64_t c = c0 + l * VEC; c < c1; c += TPT * VEC) {
      if (c + VEC <= c1) {
        if (c >= c0 + TPT * VEC) load(c);
        for (int j = 0; j < a.k; ++j)
          if (p[j] >= 0) E::template store<NT>(a.out, p[j] * a.h + c, raw[0]);
      } else {
        for (int64_t i = c; i < c1; ++i)
          for (int j = 0; j < a.k; ++j)
            if (p[j] >= 0) E::copy(a.out, p[j] * a.h + i, a.x, row * a.h + i);
      }
    }
  }
}

// out[t] = sum_j w y[inv] (+ add): a wave per token and 64 vectors of columns, U rows in flight (as
// many as k: 4096 tokens of 2048, k = 2, 8 in flight 13.6 us, 2 9.5).  NT: rows larger than the
// last-level cache are read past it (4096 tokens of 7168, k = 8: 105 -> 91 us; of 2048, k = 2, which
// the cache holds, 10.0 -> 11.0).  Where a rank holds an eighth of the slots of 4096 tokens of 7168,
// k = 8, 41 us (24 for the bytes): a row that is left out costs its vector instructions all the same,
// and these take 77 % of the cycles.
template <int DT, int U, bool NT>
__global__ void __launch_bounds__(kThreads) k_tokens_combine(const void* __restrict__ y, const int32_t* __restrict__ inv,
                                                             const float* __restrict__ w, const void* __restrict__ add,
                                                             int64_t t, int32_t k, int64_t h, uint32_t chunks,
                                                             void* __restrict__ out) {
  typedef Elem<DT> E;
  const uint32_t item = blockIdx.x * (kThreads / 64) + __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  const int64_t tok = item / chunks;
  if (tok >= t) return;
  const int64_t c = (int64_t(item - uint32_t(tok) * chunks) * 64 + (threadIdx.x & 63)) * E::VEC;
  if (c >= h) return;
  const int32_t* p = inv + tok * k;
  const float* wt = w ? w + tok * k : nullptr;
  const uint32_t rows = uint32_t(t * k);
  float acc[E::VEC];
#pragma unroll
  for (int i = 0; i < E::VEC; ++i) acc[i] = 0.f;
  const bool whole = c + E::VEC <= h;
  for (int j0 = 0; j0 < k; j0 += U) {
    int64_t at[U];
    bool ok[U];
    float wj[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = min(j0 + u, k - 1);
      const uint32_t r = uint32_t(p[j]);
      ok[u] = j0 + u < k && r < rows;   // (a dropped slot is -1 and left out)
      at[u] = int64_t(ok[u] ? r : 0) * h + c;
      wj[u] = wt ? wt[j] : 1.f;
    }
    typename E::Raw v[U];
    if (whole) {
#pragma unroll
      for (int u = 0; u < U; ++u) {   // (one branch of the whole wave: 4096 tokens of 7168, one slot of 8 held, 51 -> 45 us)
        if (ok[u]) v[u] = E::template load<NT>(y, at[u]);
        else v[u] = typename E::Raw{};
      }
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float e[E::VEC];
#pragma unroll
        for (int i = 0; i < E::VEC; ++i) e[i] = c + i < h ? E::get(y, at[u] + i) : 0.f;
        v[u] = E::pack(e);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < E::VEC; ++i) acc[i] = ok[u] ? __builtin_fmaf(wj[u], E::value(v[u], i), acc[i]) : acc[i];
  }
  const int64_t o = tok * h + c;
  if (whole) {
    if (add) {
      const typename E::Raw v = E::load(add, o);
#pragma unroll
      for (int i = 0; i < E::VEC; ++i) acc[i] += E::value(v, i);
    }
    E::store(out, o, E::pack(acc));
  } else {
#pragma unroll
    for (int i = 0; i < E::VEC; ++i)
      if (c + i < h) E::put(out, o + i, acc[i] + (add ? E::get(add, o + i) : 0.f));
  }
}

// dy and dw of a slot by TPS threads (a wave, or the workgroup where there are few slots).  NT: y and
// dy larger than the last-level cache pass it by (4096 tokens of 7168, k = 8: 207 -> 190 us; 2048
// wide, k = 2, 14.7 -> 17.1).
template <int DT, int TPS, bool NT>
__global__ void __launch_bounds__(kThreads) k_tokens_combine_bwd(const void* __restrict__ dout,
                                                                 const void* __restrict__ y,
                                                                 const int32_t* __restrict__ inv,
                                                                 const float* __restrict__ w, int64_t slots, int32_t k,
                                                                 int64_t h, void* __restrict__ dy,
                                                                 float* __restrict__ dw) {
  typedef Elem<DT> E;
  __shared__ float part[kThreads / 64];
  const int wid = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  const int64_t slot = TPS == 64 ? int64_t(blockIdx.x) * (kThreads / 64) + wid : int64_t(blockIdx.x);
  if (slot >= slots) return;
  const int l = threadIdx.x % TPS;
  const uint32_t at = uint32_t(inv[slot]);
  const float ws = w ? w[slot] : 1.f;
  const int64_t d0 = (slot / k) * h, y0 = int64_t(at) * h;
  const bool held = at < uint32_t(slots);
  float dot = 0.f;
  if (held) {
#pragma unroll 4
    for (int64_t c = l * E::VEC; c < h; c += TPS * E::VEC) {
      if (c + E::VEC <= h) {
        const typename E::Raw d = E::load(dout, d0 + c);
        if (dw) {
          const typename E::Raw v = E::template load<NT>(y, y0 + c);
#pragma unroll
          for (int i = 0; i < E::VEC; ++i) dot = __builtin_fmaf(E::value(d, i), E::value(v, i), dot);
        }
        float g[E::VEC];
#pragma unroll
        for (int i = 0; i < E::VEC; ++i) g[i] = ws * E::value(d, i);
        E::template store<NT>(dy, y0 + c, E::pack(g));
      } else {
        for (int64_t i = c; i < h; ++i) {
          const float d = E::get(dout, d0 + i);
          if (dw) dot = __builtin_fmaf(d, E::get(y, y0 + i), dot);
          E::put(dy, y0 + i, ws * d);
        }
      }
    }
  }
  if (!dw) return;
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) dot += __shfl_xor(dot, o, 64);
  if constexpr (TPS == 64) {
    if (l == 0) dw[slot] = held ? dot : 0.f;
  } else {
    if ((threadIdx.x & 63) == 0) part[wid] = dot;
    __syncthreads();
    if (threadIdx.x == 0) dw[slot] = held ? part[0] + part[1] + part[2] + part[3] : 0.f;
  }
}

template <bool QUANT, int DT, int TPW, bool NT>
hipError_t dispatch_as(const DispatchArgs& a, const int32_t* base, hipStream_t st) {
  const int64_t per = range_tokens(a.t, a.k), nr = ranges(a.t, a.k);
  const int64_t groups = (per + TPW - 1) / TPW;
  // columns over workgroups where the tokens alone do not fill the chip
  const int64_t unit = kThreads / TPW * (QUANT ? 8 : Elem<DT>::VEC);
  const int64_t most = (a.h + unit - 1) / unit;
  const int64_t split = std::max<int64_t>(1, std::min<int64_t>(most, 512 / std::max<int64_t>(1, nr * groups)));
  const int64_t block = (most + split - 1) / split * unit;
  const size_t lds = std::max<size_t>(size_t(TPW) * a.k * 4 + size_t(per) * a.k * 2, base ? 0 : size_t(a.e + 1) * 4);
  const dim3 grid(unsigned(nr * groups + (base ? 0 : 1)), unsigned((a.h + block - 1) / block));
  hipLaunchKernelGGL((k_dispatch<QUANT, DT, TPW, NT>), grid, dim3(kThreads), lds, st, a, per, base, block);
  return hipGetLastError();
}

template <bool QUANT, int DT>
hipError_t dispatch_rows(const DispatchArgs& a, const int32_t* base, hipStream_t st) {
  if (dispatch_by_waves(a.t, a.k, a.h * Elem<DT>::SIZE)) return dispatch_as<QUANT, DT, 4, false>(a, base, st);
  if (!QUANT && a.t * a.k * a.h * Elem<DT>::SIZE > kCacheBytes) return dispatch_as<QUANT, DT, 1, !QUANT>(a, base, st);
  return dispatch_as<QUANT, DT, 1, false>(a, base, st);
}

}  // namespace

int64_t dispatch_workspace(int64_t t, int32_t k, int32_t e) {
  return t * k <= kOneRange ? 0 : ranges(t, k) * (e + 1) * 4;
}

hipError_t launch_dispatch(const DispatchArgs& a, void* work, hipStream_t st) {
  int32_t* base = nullptr;
  if (a.t * a.k > kOneRange) {
    base = static_cast<int32_t*>(work);
    const int64_t per = range_tokens(a.t, a.k), nr = ranges(a.t, a.k);
    const size_t lds = size_t(a.e + 1) * 4;
    hipLaunchKernelGGL(k_order_count, dim3(unsigned(nr)), dim3(kThreads), lds, st, a.ids, a.t, a.k, a.first, a.e, per,
                       base);
    const int parts = int(std::max<int64_t>(1, std::min<int64_t>((nr + 7) / 8, 1024 / (a.e + 1))));
    hipLaunchKernelGGL(k_order_plan, dim3(1), dim3(1024), lds * (parts + 1), st, base, int(nr), a.e, parts, a.offsets);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.q) {
    if (a.dtype == 0) return dispatch_rows<true, 0>(a, base, st);
    return a.dtype == 1 ? dispatch_rows<true, 1>(a, base, st) : dispatch_rows<true, 2>(a, base, st);
  }
  // (rows are copied bit by bit: one kernel for both 16-bit types)
  return a.dtype == 0 ? dispatch_rows<false, 0>(a, base, st) : dispatch_rows<false, 1>(a, base, st);
}

hipError_t launch_tokens_combine(const void* y, const int32_t* inv, const float* w, const void* add, int64_t t,
                                 int32_t k, int64_t h, int dtype, void* out, hipStream_t st) {
  const int64_t per = 64 * (dtype == 0 ? 4 : 8), chunks = (h + per - 1) / per;
  const dim3 grid(unsigned((t * chunks + kThreads / 64 - 1) / (kThreads / 64)));
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, grid, dim3(kThreads), 0, st, y, inv, w, add, t, k, h, uint32_t(chunks), out);
    return hipGetLastError();
  };
  const bool nt = t * k * h * (dtype == 0 ? 4 : 2) > kCacheBytes;
  auto by_rows = [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    if (nt) return k <= 2 ? go(k_tokens_combine<DT, 2, true>) : k <= 4 ? go(k_tokens_combine<DT, 4, true>)
                                                                       : go(k_tokens_combine<DT, 8, true>);
    return k <= 2 ? go(k_tokens_combine<DT, 2, false>) : k <= 4 ? go(k_tokens_combine<DT, 4, false>)
                                                                : go(k_tokens_combine<DT, 8, false>);
  };
  return dtype == 0 ? by_rows(std::integral_constant<int, 0>{}) : dtype == 1 ? by_rows(std::integral_constant<int, 1>{})
                                                                             : by_rows(std::integral_constant<int, 2>{});
}

template <int TPS, bool NT>
static hipError_t combine_bwd_as(const void* dout, const void* y, const int32_t* inv, const float* w, int64_t slots,
                                 int32_t k, int64_t h, int dtype, void* dy, float* dw, hipStream_t st) {
  const dim3 grid(unsigned(TPS == 64 ? (slots + 3) / 4 : slots));
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, grid, dim3(kThreads), 0, st, dout, y, inv, w, slots, k, h, dy, dw);
  };
  if (dtype == 0) go(k_tokens_combine_bwd<0, TPS, NT>);
  else if (dtype == 1) go(k_tokens_combine_bwd<1, TPS, NT>);
  else go(k_tokens_combine_bwd<2, TPS, NT>);
  return hipGetLastError();
}

hipError_t launch_tokens_combine_bwd(const void* dout, const void* y, const int32_t* inv, const float* w, int64_t t,
                                     int32_t k, int64_t h, int dtype, void* dy, float* dw, hipStream_t st) {
  const int64_t slots = t * k;
  if (slots < 2048) return combine_bwd_as<kThreads, false>(dout, y, inv, w, slots, k, h, dtype, dy, dw, st);
  return slots * h * (dtype == 0 ? 4 : 2) > kCacheBytes
             ? combine_bwd_as<64, true>(dout, y, inv, w, slots, k, h, dtype, dy, dw, st)
             : combine_bwd_as<64, false>(dout, y, inv, w, slots, k, h, dtype, dy, dw, st);
}

}  // namespace q4
