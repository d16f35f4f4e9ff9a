// Groups of values as E4M3 codes with one fp32 scale: with a = max(the group's
// largest |v|, 2^-100), scale = a / 448 and code = E4M3(v * (448 / a)), each of
// the two quotients and the product rounded to fp32, the code to the nearest
// even.  The floor keeps 448 / a finite, so a group of zeros has codes of zero;
// an infinity or NaN makes its group's scale and codes such that every product
// with them is NaN.
#pragma once
#include "elem.h"

typedef float f32x8_t __attribute__((ext_vector_type(8)));

// Order of |v| as integers: NaN above infinity above every finite value.
DEV uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

struct GroupScale {
  float inv, scale;
};
DEV GroupScale group_scale(uint32_t amax) {
  const float a = __uint_as_float(max(amax, (127u - 100u) << 23));
  return GroupScale{448.0f / a, a / 448.0f};
}

// Four codes; |v * inv| passes 448 by rounding only, never to the next value.
DEV uint32_t codes4(float a, float b, float c, float d, float inv) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, w, true);
}

// Largest value over the lane's row of 16 lanes, in all of them.
DEV uint32_t row16_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xf, 0xf, false));   // rotated by 8
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xf, 0xf, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xf, 0xf, false));
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xf, 0xf, false));
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
