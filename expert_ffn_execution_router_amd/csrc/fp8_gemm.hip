// Products of E4M3 codes with a scale for each 128 of the summed axis.
//
//   rows:   out[r, n] = sum_g sa[g, r] sw[n / 128, g] sum_{k in group g} a[r, k] w[n, k]
//   depth:  dw[n, k]  = sum_G sdy[G, n] sx[G, k] sum_{t in group G} dy[t, n] x[t, k]
//
// In both a row operand P (a, dy transposed) with a scale per row and group
// meets a column operand Q (w, x transposed) with a scale per block of 128 or
// per column and group; both are summed along their contiguous axis.
#include "e4m3.h"
#include "op_host.h"
#include "segments.h"

namespace {

struct MmArgs {
  const uint8_t* p;            // [R][ldk] codes
  const float* sp;             // [groups][R]
  const uint8_t* q;            // [E][C][ldk] codes (depth: [C][ldk])
  const float* sq;             // blocks: [E][ceil(C/128)][groups]; depth: [groups][C]
  const int32_t* offsets;      // segments of rows, or (depth) of the summed axis; null: one
  const int32_t* counts;
  int E;
  int64_t R;
  int64_t C;
  int64_t ldk;                 // 128 * groups
  int groups;
  void* out;                   // rows: [R][ldo]; depth: [E][R][ldo]
  int64_t ldo;
  int otype, add;
};

// 8 codes as fp16, exactly.
DEV f16x8_t codes_f16(int lo, int hi) {
  const i32x4_t v = {__builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((uint32_t)lo, 1.0f, false)),
                     __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((uint32_t)lo, 1.0f, true)),
                     __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((uint32_t)hi, 1.0f, false)),
                     __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((uint32_t)hi, 1.0f, true))};
  return __builtin_bit_cast(f16x8_t, v);
}

DEV void store_value(void* out, int64_t at, int otype, float v) {
  if (otype == MOE_T_F32) ((float*)out)[at] = v;
  else if (otype == MOE_T_BF16) ((uint16_t*)out)[at] = Elem<MOE_T_BF16>::store(v);
  else ((uint16_t*)out)[at] = Elem<MOE_T_F16>::store(v);
}

constexpr int SB = 32;         // rows of a workgroup's tile

// A wave takes 32 rows x 32 columns.  The matrix instruction's columns are
// rows of P and its rows columns of Q, so a lane ends with four neighbours of
// one row.  Its sum of 8-bit codes keeps too few bits (measured: 2^-16 of the
// sum of magnitudes where values are spread), so the codes are multiplied as
// fp16, which is exact, and summed in fp32.
template <bool DEPTH>
__global__ void __launch_bounds__(256)
mm_simple_kernel(MmArgs a, int row_blocks) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, lr = lane & 15, lg = lane >> 4;
  const int64_t c0 = ((int64_t)blockIdx.x * 4 + wave) * 32;
  if (c0 >= a.C) return;
  for (int blk = blockIdx.y; blk < row_blocks; blk += gridDim.y) {
    RowBlock b{0, (int64_t)blk * SB, min((int64_t)(blk + 1) * SB, a.R)};
    int g0 = 0, g1 = a.groups;
    if (DEPTH) {
      b.e = blockIdx.z;
      if (a.offsets) {
        g0 = min(max(a.offsets[b.e], 0) / 128, a.groups);
        g1 = min(max(a.offsets[b.e + 1], 0) / 128, a.groups);
      }
    } else if (a.offsets && !find_block<SB>(a.offsets, a.counts, a.E, a.R, blk, b)) {
      return;
    }
    const uint8_t* q = a.q + (DEPTH ? 0 : b.e * a.C * a.ldk);
    const int64_t cblocks = (a.C + 127) / 128;
    const float* sq = a.sq + (DEPTH ? 0 : b.e * cblocks * a.groups);
    int64_t row[2], col[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      row[i] = min(b.at + 16 * i + lr, b.end - 1);
      col[i] = min(c0 + 16 * i + lr, a.C - 1);
    }
    f32x4_t acc[2][2] = {};
    for (int g = g0; g < g1; ++g) {
      i32x4_t pv[2][2], qv[2][2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          pv[i][h] = ld16(a.p + row[i] * a.ldk + (int64_t)g * 128 + 64 * h + 16 * lg);
          qv[i][h] = ld16(q + col[i] * a.ldk + (int64_t)g * 128 + 64 * h + 16 * lg);
        }
#pragma unroll
      for (int i = 0; i < 2; ++i) {          // columns
        float sc[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int64_t c = min(c0 + 16 * i + 4 * lg + v, a.C - 1);
          sc[v] = DEPTH ? sq[(int64_t)g * a.C + c] : sq[c / 128 * a.groups + g];
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {        // rows
          f32x4_t s = {};
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int w = 0; w < 2; ++w)
              s = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes_f16(qv[i][h][2 * w], qv[i][h][2 * w + 1]),
                                                         codes_f16(pv[j][h][2 * w], pv[j][h][2 * w + 1]), s, 0, 0, 0);
          const float sr = a.sp[(int64_t)g * a.R + row[j]];
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[i][j][v] += s[v] * (sc[v] * sr);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int64_t r = b.at + 16 * j + lr;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int64_t c = c0 + 16 * i + 4 * lg + v;
          if (r >= b.end || c >= a.C) continue;
          const int64_t at = (DEPTH ? b.e * a.R + r : r) * a.ldo + c;
          float x = acc[i][j][v];
          if (DEPTH && a.add) x += ((const float*)a.out)[at];
          store_value(a.out, at, a.otype, x);
        }
      }
  }
}

constexpr int64_t MAX_SIZE = 1 << 30, MAX_MATRIX = (int64_t)1 << 40;

}  // namespace

extern "C" {

int moe_fp8_matmul(const uint8_t* a, const float* a_scales, const int32_t* offsets, const int32_t* counts, int64_t E,
                   int64_t rows, const uint8_t* w, const float* w_scales, int64_t N, int64_t K, int otype, void* out,
                   int64_t ldo, void* stream) {
  const int b = elem_bytes(otype);
  if (!b) return bad(MOE_E_INVAL, "unknown type");
  if (rows < 0 || rows > I32_MAX) return bad(MOE_E_INVAL, "rows outside [0, 2^31)");
  if (E < 1 || E > 1024) return bad(MOE_E_INVAL, "need 1 <= E <= 1024");
  if (N < 1 || K < 1 || K % 128) return bad(MOE_E_INVAL, "need N >= 1 and K a multiple of 128");
  if (N > MAX_SIZE || K > MAX_SIZE) return bad(MOE_E_UNSUPPORTED, "more than 2^30 rows or columns");
  if (N * K > MAX_MATRIX) return bad(MOE_E_UNSUPPORTED, "a matrix of more than 2^40 values");
  if (!offsets && (E != 1 || counts)) return bad(MOE_E_INVAL, "without offsets: one matrix and no counts");
  if (ldo < N) return bad(MOE_E_INVAL, "out's row stride smaller than its width");
  if (rows == 0) return MOE_OK;
  if (!a || !a_scales || !w || !w_scales || !out) return bad(MOE_E_INVAL, "null argument");
  if (((uintptr_t)a | (uintptr_t)w) % 16) return bad(MOE_E_INVAL, "codes start on 16 bytes");
  const int64_t G = K / 128;
  if (outputs_shared({row_span(out, rows, N, ldo, b)},
                     {span(a, rows * K), span(a_scales, G * rows * 4), span(offsets, (E + 1) * 4), span(counts, E * 4),
                      span(w, E * N * K), span(w_scales, E * ((N + 127) / 128) * G * 4)}))
    return shared();
  const MmArgs m{a, a_scales, w, w_scales, offsets, counts, (int)E, rows, N, K, (int)G, out, ldo, otype, 0};
  // blocks of the segments: one more than the rows fill at most for each expert that has rows
  const int64_t blocks = (rows + SB - 1) / SB + (offsets ? std::min(E, rows) : 0);
  const dim3 grid((unsigned)((N + 127) / 128), (unsigned)std::min<int64_t>(blocks, 65535));
  mm_simple_kernel<false><<<grid, 256, 0, (hipStream_t)stream>>>(m, (int)blocks);
  return launched();
}

int moe_fp8_weight_gradient(const uint8_t* dy_t, const float* dy_scales, const uint8_t* x_t, const float* x_scales,
                            const int32_t* offsets, int64_t E, int64_t rows, int64_t N, int64_t K, int add, float* dw,
                            int64_t ldw, void* stream) {
  if (rows < 0 || rows > I32_MAX) return bad(MOE_E_INVAL, "rows outside [0, 2^31)");
  if (E < 1 || E > 1024) return bad(MOE_E_INVAL, "need 1 <= E <= 1024");
  if (!offsets && E != 1) return bad(MOE_E_INVAL, "without offsets: one matrix");
  if (N < 1 || K < 1) return bad(MOE_E_INVAL, "need N >= 1 and K >= 1");
  if (N > MAX_SIZE || K > MAX_SIZE || rows > MAX_SIZE) return bad(MOE_E_UNSUPPORTED, "more than 2^30 rows or columns");
  if (N * K > MAX_MATRIX) return bad(MOE_E_UNSUPPORTED, "a matrix of more than 2^40 values");
  if (ldw < K) return bad(MOE_E_INVAL, "dw's row stride smaller than its width");
  if (ldw > ((int64_t)1 << 40)) return bad(MOE_E_UNSUPPORTED, "dw's row stride over 2^40");
  if (!dw || (rows && (!dy_t || !dy_scales || !x_t || !x_scales))) return bad(MOE_E_INVAL, "null argument");
  if (((uintptr_t)dy_t | (uintptr_t)x_t) % 16) return bad(MOE_E_INVAL, "codes start on 16 bytes");
  const int64_t Rp = (rows + 127) / 128 * 128, G = Rp / 128;
  if (outputs_shared({row_span(dw, E * N, K, ldw, 4)},
                     {span(dy_t, N * Rp), span(dy_scales, G * N * 4), span(x_t, K * Rp), span(x_scales, G * K * 4),
                      span(offsets, (E + 1) * 4)}))
    return shared();
  const MmArgs m{dy_t, dy_scales, x_t, x_scales, offsets, nullptr, (int)E, N, K, Rp, (int)G, dw, ldw, MOE_T_F32, add};
  const int64_t blocks = (N + SB - 1) / SB;
  const dim3 grid((unsigned)((K + 127) / 128), (unsigned)std::min<int64_t>(blocks, 65535), (unsigned)E);
  mm_simple_kernel<true><<<grid, 256, 0, (hipStream_t)stream>>>(m, (int)blocks);
  return launched();
}

}  // extern "C"
