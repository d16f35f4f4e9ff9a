// Values of the element types in and out of registers.
#pragma once
#include "common.h"
#include "moe.h"

template <int DT>
struct Elem;
template <>
struct Elem<MOE_T_BF16> {
  typedef uint16_t type;
  static DEV float load(uint16_t v) { return bf16_bits_to_f32(v); }
  static DEV uint16_t store(float v) { return (uint16_t)pack_bf16x2(v, 0.0f); }
};
template <>
struct Elem<MOE_T_F16> {
  typedef uint16_t type;
  static DEV float load(uint16_t v) { return (float)__builtin_bit_cast(_Float16, v); }
  static DEV uint16_t store(float v) { return (uint16_t)pack_f16x2(v, 0.0f); }
};
template <>
struct Elem<MOE_T_F32> {
  typedef float type;
  static DEV float load(float v) { return v; }
  static DEV float store(float v) { return v; }
};

// V values, aligned as one is.
template <typename T, int V>
struct Pack {
  T v[V];
};

template <int DT, int V>
DEV void load_vals(const typename Elem<DT>::type* p, float (&f)[V]) {
  Pack<typename Elem<DT>::type, V> a;
  __builtin_memcpy(&a, p, sizeof(a));
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = Elem<DT>::load(a.v[i]);
}

template <int DT, int V>
DEV void store_vals(typename Elem<DT>::type* p, const float (&f)[V]) {
  Pack<typename Elem<DT>::type, V> a;
#pragma unroll
  for (int i = 0; i < V; ++i) a.v[i] = Elem<DT>::store(f[i]);
  __builtin_memcpy(p, &a, sizeof(a));
}
