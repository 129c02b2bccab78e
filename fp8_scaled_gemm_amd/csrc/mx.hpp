// Device helpers of the microscaled formats: MXFP4 matrices (mxfp4_operand in
// the C ABI) and 8-bit activation checkpoints (fp8sg_act8).
//
// A block of 32 values shares one power of two 2^(s - 127).  Its exponent comes
// from the bits of the block's largest magnitude, and dividing by a power of
// two is exact, so quantising needs no rounding but the element's own: the
// gfx950 converts take the scale as an operand, divide by it and round to
// nearest even with saturation (checked over every bf16 and fp16 value and
// scales from 2^-127 to 2^125 against the definition).
#pragma once

#include <utility>

#include "common.hpp"
#include "launch_mx.hpp"

namespace fp8sg {

// f(integral constants 0 .. N - 1): a loop whose index is a constant expression
template <int... I, class F>
__device__ __forceinline__ void static_for_(std::integer_sequence<int, I...>, F f) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void static_for(F f) {
  static_for_(std::make_integer_sequence<int, N>{}, f);
}

// ---- element types (fp8sg_out values)
template <int T>
struct ElemOf { typedef uint16_t type; };
template <>
struct ElemOf<FP8SG_OUT_F32> { typedef float type; };
template <int T>
using Elem = typename ElemOf<T>::type;

// fp32 -> element, rounded once to nearest even
template <int T>
__device__ __forceinline__ Elem<T> from_f32(float v) {
  if constexpr (T == FP8SG_OUT_BF16) return __builtin_bit_cast(uint16_t, (__bf16)v);
  else if constexpr (T == FP8SG_OUT_F16) return __builtin_bit_cast(uint16_t, (_Float16)fp32_value(v));
  else return v;
}

// ---- block scales
// Scale byte of a block whose largest magnitude has the fp32 bits `amax` (sign
// cleared): floor(log2 amax) is the exponent field, so floor(log2 amax) - emax
// + 127 = field - emax.  `fit` raises it by one where the mantissa exceeds the
// largest element's (kMant: 1.5 for e2m1's 6, 1.75 for e4m3's 448), up to
// 254 - emax, where the largest element times the scale is still finite
// (floor never exceeds that).  Subnormal magnitudes count as field 0: both
// rules give them the smallest scale, 2^-127, of which they are below 2.
template <int EMAX, uint32_t kMant>
__device__ __forceinline__ uint32_t block_scale(uint32_t amax, bool fit) {
  if (amax >= 0x7F800000u) return 255u;
  int e = (int)(amax >> 23) - EMAX;
  if (fit && (amax & 0x7FFFFFu) > kMant) e = e + 1 < 254 - EMAX ? e + 1 : 254 - EMAX;
  return (uint32_t)(e > 0 ? e : 0);
}
__device__ __forceinline__ uint32_t fp4_scale(uint32_t amax, bool fit) {
  return block_scale<2, 0x400000u>(amax, fit);
}
__device__ __forceinline__ uint32_t act8_scale(uint32_t amax) {
  return block_scale<8, 0x600000u>(amax, true);
}
// 2^(s - 127) as fp32 (s = 0: the subnormal 2^-127); s = 255: NaN
__device__ __forceinline__ float scale_value(uint32_t s) {
  if (s == 255u) return __uint_as_float(0x7FC00000u);
  return __uint_as_float(s ? s << 23 : 0x00400000u);
}

// e4m3 codes of values in a block with scale byte s: v * 2^(127 - s) is exact
// (or far below half the smallest code), and a magnitude past 448, possible
// only where the scale is at its upper end, is clamped.
__device__ __forceinline__ float act8_inv(uint32_t s) {
  // 2^(127 - s), s in [0, 246]: exponent field 254 - s >= 8
  return __uint_as_float((254u - s) << 23);
}
__device__ __forceinline__ float act8_clamp(float v) { return fminf(fmaxf(v, -kE4M3Max), kE4M3Max); }
// Eight values of a block with scale byte s to eight codes (s = 255: zeros).
__device__ __forceinline__ uint2 act8_codes(const float (&v)[8], uint32_t s) {
  if (s == 255u) return make_uint2(0, 0);
  const float inv = act8_inv(s);
  return make_uint2(cvt4<FP8SG_E4M3FN>(act8_clamp(v[0] * inv), act8_clamp(v[1] * inv), act8_clamp(v[2] * inv),
                                       act8_clamp(v[3] * inv)),
                    cvt4<FP8SG_E4M3FN>(act8_clamp(v[4] * inv), act8_clamp(v[5] * inv), act8_clamp(v[6] * inv),
                                       act8_clamp(v[7] * inv)));
}
// Eight codes back to values.
__device__ __forceinline__ void act8_values(uint2 q, uint32_t s, float (&v)[8]) {
  const float sc = scale_value(s);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int w = (int)(h ? q.y : q.x);
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
    v[4 * h] = lo[0] * sc;
    v[4 * h + 1] = lo[1] * sc;
    v[4 * h + 2] = hi[0] * sc;
    v[4 * h + 3] = hi[1] * sc;
  }
}
// Largest of four neighbouring lanes' values, in each of them (two DPP steps;
// all four lanes active).
__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
  uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, false);
  m = o > m ? o : m;
  o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, false);
  return o > m ? o : m;
}
// Largest magnitude (fp32 bits) of the 32 values that four neighbouring lanes
// hold eight each of; every lane of the four gets it.
__device__ __forceinline__ uint32_t quad_amax(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t a = __float_as_uint(v[e]) & 0x7FFFFFFFu;
    m = a > m ? a : m;
  }
  return quad_max(m);
}

// ---- eight consecutive elements of a row, p[0 .. 7], of which n are in range
// (the rest read as 0 and are not written).  Whole groups move as 16-byte
// accesses at whatever address the row has: the hardware takes any, and the
// type tells the compiler.  S: non-temporal.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
template <bool S>
__device__ __forceinline__ u32x4 ld_any(const void* p) {
  const u32x4_any* q = reinterpret_cast<const u32x4_any*>(p);
  const u32x4_any v = S ? __builtin_nontemporal_load(q) : *q;
  return u32x4{v.x, v.y, v.z, v.w};
}
template <bool S>
__device__ __forceinline__ void st_any(void* p, u32x4 v) {
  u32x4_any* q = reinterpret_cast<u32x4_any*>(p);
  const u32x4_any w = {v.x, v.y, v.z, v.w};
  if constexpr (S) __builtin_nontemporal_store(w, q);
  else *q = w;
}

// As loaded: 4 dwords of 16-bit elements or 8 of fp32.
template <int T>
struct Row8 {
  static constexpr int kW = T == FP8SG_OUT_F32 ? 8 : 4;
  uint32_t w[kW];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kW; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (T == FP8SG_OUT_F32) v[e] = __uint_as_float(w[e]);
      else v[e] = (e & 1) ? in_hi<T == FP8SG_OUT_F16>(w[e / 2]) : in_lo<T == FP8SG_OUT_F16>(w[e / 2]);
    }
  }
};
template <int T, bool S>
__device__ __forceinline__ Row8<T> load_row8(const Elem<T>* p, int n) {
  Row8<T> r;
  if (n >= 8) {
#pragma unroll
    for (int h = 0; h < Row8<T>::kW / 4; ++h) {
      const u32x4 v = ld_any<S>(p + 4 * h);
      r.w[4 * h] = v.x;
      r.w[4 * h + 1] = v.y;
      r.w[4 * h + 2] = v.z;
      r.w[4 * h + 3] = v.w;
    }
  } else {  // the row's end, element by element (constant offsets: nothing for a loop around it to keep)
    r.zero();
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (e < n) {
        if constexpr (T == FP8SG_OUT_F32) r.w[e] = __float_as_uint(p[e]);
        else r.w[e / 2] |= (uint32_t)p[e] << (16 * (e & 1));
      }
    }
  }
  return r;
}
template <int T, bool S>
__device__ __forceinline__ void load8(const Elem<T>* p, int n, float (&v)[8]) {
  load_row8<T, S>(p, n).values(v);
}
template <int T, bool S>
__device__ __forceinline__ void store8(Elem<T>* p, int n, const float (&v)[8]) {
  if (n >= 8) {
    if constexpr (T == FP8SG_OUT_F32) {
      st_any<S>(p, u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])});
      st_any<S>(p + 4, u32x4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])});
    } else {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = (uint32_t)from_f32<T>(v[2 * e]) | ((uint32_t)from_f32<T>(v[2 * e + 1]) << 16);
      st_any<S>(p, u32x4{w[0], w[1], w[2], w[3]});
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) p[e] = from_f32<T>(v[e]);
  }
}
// elements of the 8 from c on that a row of `cols` has
__device__ __forceinline__ int left8(int64_t cols, int64_t c) { return cols - c < 8 ? (int)(cols - c) : 8; }

}  // namespace fp8sg
