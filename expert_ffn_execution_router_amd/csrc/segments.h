// Row blocks of grouped rows, found on the device from the segments.
#pragma once
#include "common.h"

// A block of up to BM rows of one expert.
struct RowBlock {
  int e;
  int64_t at, end;
};

// The want-th block in expert order; false if there are fewer.  Every wave
// finds it for itself: 64 experts at a time, a wave scan counts their blocks.
// Segments are cut to the rows there are.
template <int BM>
DEV bool find_block(const int32_t* __restrict__ offsets, const int32_t* __restrict__ counts, int E, int64_t rows,
                    int want, RowBlock& b) {
  const int lane = threadIdx.x & 63;
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = min(e0 + lane, E - 1);
    const int64_t first = offsets[e];
    const int64_t many = counts ? (int64_t)counts[e] : offsets[e + 1] - first;
    const int64_t at = min(max(first, (int64_t)0), rows), end = min(max(first + many, at), rows);
    const int mine = e0 + lane < E ? (int)((end - at + BM - 1) / BM) : 0;
    int sum = mine;                                   // blocks of this lane's expert and those before it
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(sum, d, 64);
      if (lane >= d) sum += v;
    }
    const int all = __shfl(sum, 63, 64);
    if (want < all) {
      const uint64_t m = __builtin_amdgcn_ballot_w64(sum > want);
      const int who = __builtin_ctzll(m);
      const int k = want - __shfl(sum - mine, who, 64);
      const int64_t a = __shfl(at, who, 64), z = __shfl(end, who, 64);
      b.e = e0 + who;
      b.at = a + (int64_t)k * BM;
      b.end = min(b.at + BM, z);
      return true;
    }
    want -= all;
  }
  return false;
}
