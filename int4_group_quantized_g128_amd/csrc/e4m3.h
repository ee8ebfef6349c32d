// e4m3 codes (OCP, largest 448) with one fp32 scale per group, and elements of the float types.
#pragma once
#include "common.h"

namespace q4 {

constexpr int kE4m3Group = 128;
constexpr float kE4m3Max = 448.f;

// Elements of dtype DT (0 fp32, 1 fp16, 2 bf16) and vectors of 16 bytes of them, at any element's
// address: the target's global accesses need no alignment.
template <int DT> struct Elem {
  static constexpr int SIZE = DT == 0 ? 4 : 2;
  static constexpr int VEC = 16 / SIZE;
  static Q4_DEVICE float get(const void* p, int64_t i) {
    if constexpr (DT == 0) return static_cast<const float*>(p)[i];
    else if constexpr (DT == 1) return f16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
    else return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
  }
  static Q4_DEVICE void put(void* p, int64_t i, float v) {
    if constexpr (DT == 0) static_cast<float*>(p)[i] = v;
    else if constexpr (DT == 1) static_cast<uint16_t*>(p)[i] = bitcast<uint16_t>(_Float16(v));
    else static_cast<uint16_t*>(p)[i] = bitcast<uint16_t>(__bf16(v));
  }
  static Q4_DEVICE void copy(void* to, int64_t i, const void* from, int64_t j) {   // the bits, NaNs too
    if constexpr (DT == 0) static_cast<uint32_t*>(to)[i] = static_cast<const uint32_t*>(from)[j];
    else static_cast<uint16_t*>(to)[i] = static_cast<const uint16_t*>(from)[j];
  }
  struct __attribute__((packed, aligned(SIZE))) Raw {
    uint32_t w[4];
  };
  template <bool NT = false>
  static Q4_DEVICE Raw load(const void* p, int64_t i) {
    const uint8_t* at = static_cast<const uint8_t*>(p) + i * SIZE;
    if constexpr (NT) {
      typedef u32x4_t any_t __attribute__((aligned(2)));
      return bitcast<Raw>(u32x4_t(__builtin_nontemporal_load(reinterpret_cast<const any_t*>(at))));
    }
    return *reinterpret_cast<const Raw*>(at);
  }
  template <bool NT = false>
  static Q4_DEVICE void store(void* p, int64_t i, const Raw& r) {
    uint8_t* at = static_cast<uint8_t*>(p) + i * SIZE;
    if constexpr (NT) {
      typedef u32x4_t any_t __attribute__((aligned(2)));
      __builtin_nontemporal_store(bitcast<u32x4_t>(r), reinterpret_cast<any_t*>(at));
    } else {
      *reinterpret_cast<Raw*>(at) = r;
    }
  }
  static Q4_DEVICE float value(const Raw& r, int i) {
    if constexpr (DT == 0) return __uint_as_float(r.w[i]);
    const uint16_t h = uint16_t(r.w[i / 2] >> (16 * (i % 2)));
    return DT == 1 ? f16_bits_to_f32(h) : bf16_to_f32(h);
  }
  static Q4_DEVICE Raw pack(const float* v) {
    Raw r;
    if constexpr (DT == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) r.w[i] = __float_as_uint(v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint16_t a, b;
        if constexpr (DT == 1) a = bitcast<uint16_t>(_Float16(v[2 * i])), b = bitcast<uint16_t>(_Float16(v[2 * i + 1]));
        else a = bitcast<uint16_t>(__bf16(v[2 * i])), b = bitcast<uint16_t>(__bf16(v[2 * i + 1]));
        r.w[i] = a | uint32_t(b) << 16;
      }
    }
    return r;
  }
};

// |v| for a group's largest magnitude: a NaN becomes an infinity, which no finite value does.
Q4_DEVICE float magnitude(float v) {
  const float a = fabsf(v);
  return a == a ? a : __builtin_inff();
}

// Largest of 16 lanes (a DPP row) in every one of them.
template <int CTRL>
Q4_DEVICE float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, false));
}
Q4_DEVICE float row16_max(float v) {
  v = fmaxf(v, dpp<0xB1>(v));    // quad_perm [1, 0, 3, 2]
  v = fmaxf(v, dpp<0x4E>(v));    // quad_perm [2, 3, 0, 1]
  v = fmaxf(v, dpp<0x141>(v));   // row_half_mirror
  return fmaxf(v, dpp<0x140>(v));   // row_mirror
}

// x / s rounded once, for 2^-80 <= s: r is 1 / s rounded once.  Two steps of the remainder, each
// exact in one fma, leave an error before the last rounding below the distance of any quotient of
// two fp32 numbers from a tie (5 operations where the general division takes 11 and a reciprocal;
// codes along rows and tokens of 4096 x 16384 bf16 90 -> 77 us).  Quotients below 2^-11, whose code
// is 0 either way, may be off.
constexpr float kPlainScale = 0x1p-80f;
Q4_DEVICE float quotient(float x, float s, float r) {
  float q = x * r;
  q = __builtin_fmaf(__builtin_fmaf(-q, s, x), r, q);
  return __builtin_fmaf(__builtin_fmaf(-q, s, x), r, q);
}

// Scale of a group with largest magnitude m: m / 448 (IEEE), NaN for a group with an infinity or
// a NaN (its codes are 0, so that every result that it enters is NaN).
Q4_DEVICE float e4m3_scale(float m) {
  if (m >= 0x1p-60f) return m < __builtin_inff() ? quotient(m, kE4m3Max, 1.f / kE4m3Max) : __builtin_nanf("");
  return m / kE4m3Max;
}

Q4_DEVICE uint32_t e4m3_pack4(float a, float b, float c, float d) {
  const int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true));
}

// Eight codes: e4m3 of v / s (IEEE quotient, then half to even), 0 where s is 0 or NaN.  (The clamp
// is for quotients that round past 448 and scales below fp32's normal range.)
Q4_DEVICE float e4m3_clamp(float q) { return __builtin_amdgcn_fmed3f(q, -kE4m3Max, kE4m3Max); }
Q4_DEVICE u32x2_t e4m3_codes8(const float* v, float s) {
  if (!(s > 0.f)) return u32x2_t{0, 0};
  float c[8];
  if (s >= kPlainScale) {
    const float r = 1.f / s;
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = e4m3_clamp(quotient(v[i], s, r));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = e4m3_clamp(v[i] / s);
  }
  return u32x2_t{e4m3_pack4(c[0], c[1], c[2], c[3]), e4m3_pack4(c[4], c[5], c[6], c[7])};
}

}  // namespace q4
