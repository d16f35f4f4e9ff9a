// Internal (not part of the C ABI): host check that a call's outputs share no
// memory with its inputs or with each other.
#pragma once
#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

// n runs of `bytes`, `stride` bytes from one's start to the next's.
struct Span {
  const void* at;
  int64_t n, bytes;
  __int128 stride;
};

inline Span span(const void* p, int64_t bytes) { return Span{p, 1, bytes, 0}; }

// Rows of cols values, ld values apart.
inline Span row_span(const void* p, int64_t rows, int64_t cols, int64_t ld, int value_bytes) {
  return Span{p, rows, cols * value_bytes, (__int128)ld * value_bytes};
}

// Runs of one stride (a single run has any) may interleave, as column ranges
// of one buffer do; with different strides the whole ranges are compared.
inline bool meet(const Span& a, const Span& b) {
  if (!a.at || !b.at || a.n < 1 || b.n < 1 || a.bytes < 1 || b.bytes < 1) return false;
  const __int128 a0 = (__int128)(uintptr_t)a.at, b0 = (__int128)(uintptr_t)b.at;
  if (a0 + (a.n - 1) * a.stride + a.bytes <= b0 || b0 + (b.n - 1) * b.stride + b.bytes <= a0) return false;
  if ((a.n == 1 && b.n == 1) || (a.n > 1 && b.n > 1 && a.stride != b.stride)) return true;
  const __int128 s = a.n > 1 ? a.stride : b.stride, d = ((b0 - a0) % s + s) % s;
  return d < a.bytes || d + b.bytes > s;
}

inline bool outputs_shared(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (auto o = outs.begin(); o != outs.end(); ++o) {
    for (const Span& i : ins)
      if (meet(*o, i)) return true;
    for (auto p = o + 1; p != outs.end(); ++p)
      if (meet(*o, *p)) return true;
  }
  return false;
}
