// Groups of values as E4M3 codes with one fp32 scale: with a = max(the group's
// largest |v|, 2^-100), scale = a / 448 and code = E4M3(v * (448 / a)), each of
// the two quotients and the product rounded to fp32, the code to the nearest
// even.  The floor keeps 448 / a finite, so a group of zeros has codes of zero;
// an infinity or NaN makes its group's scale and codes such that every product
// with them is NaN.
#pragma once
#include "elem.h"

typedef float f32x8_t __attribute__((ext_vector_type(8)));

// The larger; NaN if either is (of equal values, zeros of either sign).
DEV float maximum(float a, float b) { return __builtin_elementwise_maximum(a, b); }

template <int N>
DEV float abs_max(const float (&v)[N]) {
  float m = fabsf(v[0]);
#pragma unroll
  for (int i = 1; i < N; ++i) m = maximum(m, fabsf(v[i]));
  return m;
}

struct GroupScale {
  float inv, scale;
};
DEV GroupScale group_scale(float amax) {
  const float a = maximum(amax, 0x1p-100f);
  return GroupScale{448.0f / a, a / 448.0f};
}

// Four codes; |v * inv| passes 448 by rounding only, never to the next value.
DEV uint32_t codes4(float a, float b, float c, float d, float inv) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, w, true);
}

template <int CTRL>
DEV float dpp(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), CTRL, 0xf, 0xf, true));
}

// Largest value over the lane's row of 16 lanes, in all of them.
DEV float row16_max(float v) {
  v = maximum(v, dpp<0x128>(v));         // rotated by 8
  v = maximum(v, dpp<0x124>(v));
  v = maximum(v, dpp<0x122>(v));
  return maximum(v, dpp<0x121>(v));
}

// The same over lanes l, l ^ 16, l ^ 32, l ^ 48.
DEV float lanes_max(float v) {
  typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
  uint32_t b = __float_as_uint(v);
  u32x2_t p = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane16_swap(b, b, false, false));
  b = __float_as_uint(maximum(__uint_as_float(p[0]), __uint_as_float(p[1])));
  p = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane32_swap(b, b, false, false));
  return maximum(__uint_as_float(p[0]), __uint_as_float(p[1]));
}

// Lane I of the lane's quad.
template <int I>
DEV float quad_lane(float v) {
  return dpp<I * 0x55>(v);
}

// Up to 8 values from column c on; zeros from column cols on.
template <int DT>
DEV void load8(const typename Elem<DT>::type* row, long c, long cols, float (&f)[8]) {
  if (c + 8 <= cols) {
    load_vals<DT, 8>(row + c, f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = c + i < cols ? Elem<DT>::load(row[c + i]) : 0.0f;
  }
}

template <int DT>
DEV void store8(typename Elem<DT>::type* row, long c, long cols, const float (&f)[8]) {
  if (c + 8 <= cols) {
    store_vals<DT, 8>(row + c, f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < cols) row[c + i] = Elem<DT>::store(f[i]);
  }
}

DEV float silu(float g) { return g / (1.0f + expf(-g)); }
