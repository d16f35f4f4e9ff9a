// Products of a few rows with 4-bit weights in groups of consecutive inputs
// that share a 16-bit scale and (optionally) zero point, dense or per expert
// over grouped rows, optionally gated.
//
//   z[r,n] = sum_k x[r,k] (q[n,k] - zero[n,k/G]) scale[n,k/G]
//          = sum_groups scale ( sum_k x q  -  zero sum_k x )
//   gated: out = silu(z[:, :N/2]) * z[:, N/2:], else out = z
//
// With few rows the weights are each used a few times: the bound is their
// stream from HBM (N K / 2 bytes of codes).  The codes 0..15 meet x in the
// 16x16x32 matrix instruction, exactly: a nibble in a byte is the E4M3 code
// of q 2^-9 (subnormals and the first binade count up without a gap), so one
// conversion scaled by 2^9 turns two codes into two exact bf16 or fp16
// integers, and the products are exact in fp32.  The group's sum of x comes
// from one more matrix instruction with a constant operand, shared by all
// weight rows: with the default zero of 8 the constant is -8 and its result
// is where the group's sum starts, otherwise it is 1 and the zero point
// multiplies its result.  Scales then multiply fp32 sums: the only roundings
// are those of fp32 sums and of the output.
#include "common.h"
#include "fwd_ws.h"
#include "moe.h"

namespace {

struct W4Args {
  const uint16_t* x;
  long ldx, xrows;
  const int32_t* row_map;      // null: grouped row r reads x row r
  int map_div;
  const int32_t* offsets;      // null: dense, rows 0 .. rows
  const int32_t* counts;       // null: segments without padding
  int E;
  long rows;
  const uint8_t* codes;
  const uint16_t* scales;
  const uint16_t* zeros;
  int N, K, G;
  bool scale_f16;
  void* out;
  long ldo;
};

DEV float silu_mul(float g, float u) { return g / (1.0f + expf(-g)) * u; }

template <int XT>
struct Frag;
template <>
struct Frag<MOE_T_BF16> {
  typedef bf16x8_t type;
  static DEV f32x4_t mfma(type a, type b, f32x4_t c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
  static DEV uint32_t lo(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 512.0f, false));
  }
  static DEV uint32_t hi(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 512.0f, true));
  }
  static DEV float value(uint16_t b) { return bf16_bits_to_f32(b); }
  static constexpr int ONE = 0x3F803F80, MINUS8 = (int)0xC100C100;
};
template <>
struct Frag<MOE_T_F16> {
  typedef f16x8_t type;
  static DEV f32x4_t mfma(type a, type b, f32x4_t c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
  static DEV uint32_t lo(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 512.0f, false));
  }
  static DEV uint32_t hi(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 512.0f, true));
  }
  static DEV float value(uint16_t b) { return (float)__builtin_bit_cast(_Float16, b); }
  static constexpr int ONE = 0x3C003C00, MINUS8 = (int)0xC800C800;
};

// The 8 codes of a word (two per byte, even input in the low nibble) as 8
// integers in input order.
template <int XT>
DEV typename Frag<XT>::type codes8(uint32_t w) {
  const uint32_t even = w & 0x0F0F0F0Fu, odd = (w >> 4) & 0x0F0F0F0Fu;
  const uint32_t a = __builtin_amdgcn_perm(odd, even, 0x05010400u), b = __builtin_amdgcn_perm(odd, even, 0x07030602u);
  const i32x4_t v = {(int)Frag<XT>::lo(a), (int)Frag<XT>::hi(a), (int)Frag<XT>::lo(b), (int)Frag<XT>::hi(b)};
  return __builtin_bit_cast(typename Frag<XT>::type, v);
}

// 4 x 4 transpose of dwords over the wave's four 16-lane rows: word i of
// row g becomes word g of row i.
DEV void transpose_rows(i32x4_t& a) {
  const auto p = __builtin_amdgcn_permlane32_swap((uint32_t)a[0], (uint32_t)a[2], false, false);
  const auto q = __builtin_amdgcn_permlane32_swap((uint32_t)a[1], (uint32_t)a[3], false, false);
  const auto r = __builtin_amdgcn_permlane16_swap(p[0], q[0], false, false);
  const auto s = __builtin_amdgcn_permlane16_swap(p[1], q[1], false, false);
  a = i32x4_t{(int)r[0], (int)r[1], (int)s[0], (int)s[1]};
}

DEV void store_out(uint16_t* p, float v, std::integral_constant<int, MOE_T_BF16>) {
  *p = (uint16_t)pack_bf16x2(v, 0.0f);
}
DEV void store_out(uint16_t* p, float v, std::integral_constant<int, MOE_T_F16>) { *p = (uint16_t)pack_f16x2(v, 0.0f); }

// One workgroup: NR tiles of 16 weight rows (gated: NR / 2 gate tiles and
// the matching up tiles) against the rows of one expert (or of the dense
// product's row block), 16 * TT at a time.  Its waves split the inputs in
// steps of 128: wave v takes steps v, v + waves, ..., and the waves' sums are
// added through LDS in wave order.  In a step lane (g, l) of a wave (g = lane
// / 16) holds 32 codes (16 bytes) of weight row l at inputs 32 g ..; as
// operand fragment i they are inputs 32 g + 8 i .. for groups of 128 and more
// (the group spans the step, so the order of its inputs is free as long as x
// is read alike), and for smaller groups the words are exchanged between the
// lane rows so that fragment i holds inputs 32 i + 8 g ..: one fragment is
// then one run of 32 inputs.
template <int XT, int GM, int NR, int TT, bool GATED, bool HZ>
__global__ void __launch_bounds__(256)
w4_kernel(W4Args a, int otype) {
  typedef Frag<XT> F;
  typedef typename F::type frag;
  constexpr int SUB = 128 / GM;                  // groups per step
  constexpr int NO = GATED ? NR / 2 : NR;        // output tiles
  constexpr int U = TT == 1 ? 4 : (TT == 2 ? 2 : 1);
  extern __shared__ f32x4_t red[];               // [waves][NR * TT][64]
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const int g = lane >> 4, l = lane & 15;
  const int NH = GATED ? a.N / 2 : a.N;
  const int n0 = blockIdx.x * 16 * NO;
  // the rows of this workgroup
  long r_at, r_end;
  size_t e = 0;
  if (a.offsets) {
    // expert: the blockIdx.y-th one that has rows
    int want = blockIdx.y, found = 0, cnt = 0, off = 0;
    for (int e0 = 0; e0 < a.E && !found; e0 += 64) {
      const int ee = e0 + lane;
      int o = 0, c = 0;
      if (ee < a.E) {
        o = a.offsets[ee];
        c = a.counts ? a.counts[ee] : a.offsets[ee + 1] - o;
      }
      uint64_t m = __builtin_amdgcn_ballot_w64(c > 0);
      const int here = __popcll(m);
      if (want < here) {
        for (int i = 0; i < want; ++i) m &= m - 1ull;
        const int at = __builtin_ctzll(m);
        e = e0 + at;
        off = __builtin_amdgcn_readlane(o, at);
        cnt = __builtin_amdgcn_readlane(c, at);
        found = 1;
      } else {
        want -= here;
      }
    }
    if (!found) return;
    r_at = off < 0 ? 0 : off;
    r_end = (long)off + cnt;
    if (r_end > a.rows) r_end = a.rows;
  } else {
    r_at = (long)blockIdx.y * 16 * TT;
    r_end = r_at + 16 * TT < a.rows ? r_at + 16 * TT : a.rows;
  }
  const int NG = a.K / a.G, steps = (a.K + 127) / 128;
  const uint8_t* wp[NR];
  const uint16_t* sp[NR];
  const uint16_t* zp[NR];
#pragma unroll
  for (int q = 0; q < NR; ++q) {
    int n = n0 + 16 * (q % NO) + l;
    if (n >= NH) n = NH - 1;                     // loaded, not stored
    const size_t row = e * a.N + (q / NO) * NH + n;
    wp[q] = a.codes + row * (a.K / 2) + 16 * g;
    sp[q] = a.scales + row * NG;
    zp[q] = HZ ? a.zeros + row * NG : nullptr;
  }
  const i32x4_t zero4 = {0, 0, 0, 0};
  const int cst = HZ ? F::ONE : F::MINUS8;
  const frag cfrag = __builtin_bit_cast(frag, (i32x4_t){cst, cst, cst, cst});
  for (long r0 = r_at; r0 < r_end; r0 += 16 * TT) {
    const uint16_t* xr[TT];                      // this lane's x rows (null: none)
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const long r = r0 + 16 * t + l;
      xr[t] = nullptr;
      if (r < r_end) {
        const long src = a.row_map ? (a.row_map[r] < 0 ? -1 : a.row_map[r] / a.map_div) : r;
        if (src >= 0 && src < a.xrows) xr[t] = a.x + src * a.ldx;
      }
    }
    f32x4_t total[NR][TT];
#pragma unroll
    for (int q = 0; q < NR; ++q)
#pragma unroll
      for (int t = 0; t < TT; ++t) total[q][t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    for (int s0 = wave; s0 < steps; s0 += waves * U) {
      i32x4_t wv[U][NR], xv[U][TT][4];
      uint16_t sc[U][NR][SUB], zc[U][NR][SUB];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int s = s0 + u * waves;
        const bool ok = 128 * s + 32 * g < a.K;
#pragma unroll
        for (int q = 0; q < NR; ++q) {
          wv[u][q] = ok ? ld16_nt(wp[q] + (size_t)64 * s) : zero4;
#pragma unroll
          for (int h = 0; h < SUB; ++h) {
            const int k = 128 * s + GM * h;
            sc[u][q][h] = k < a.K ? sp[q][k / a.G] : 0;
            zc[u][q][h] = HZ && k < a.K ? zp[q][k / a.G] : 0;
          }
        }
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int k = 128 * s + (GM == 128 ? 32 * g + 8 * i : 32 * i + 8 * g);
            xv[u][t][i] = xr[t] && k < a.K ? ld16(xr[t] + k) : zero4;
          }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (s0 + u * waves >= steps) break;
        f32x4_t xsum[TT][SUB];
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
          for (int h = 0; h < SUB; ++h) {
            f32x4_t c = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < 4 / SUB; ++i)
              c = F::mfma(__builtin_bit_cast(frag, xv[u][t][h * (4 / SUB) + i]), cfrag, c);
            xsum[t][h] = c;
          }
#pragma unroll
        for (int q = 0; q < NR; ++q) {
          i32x4_t w = wv[u][q];
          if (GM < 128) transpose_rows(w);
          frag b[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) b[i] = codes8<XT>((uint32_t)w[i]);
#pragma unroll
          for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int h = 0; h < SUB; ++h) {
              f32x4_t c = {0.0f, 0.0f, 0.0f, 0.0f};
              if (!HZ) c = xsum[t][h];
#pragma unroll
              for (int i = 0; i < 4 / SUB; ++i)
                c = F::mfma(__builtin_bit_cast(frag, xv[u][t][h * (4 / SUB) + i]), b[h * (4 / SUB) + i], c);
              const float s = a.scale_f16 ? Frag<MOE_T_F16>::value(sc[u][q][h]) : bf16_bits_to_f32(sc[u][q][h]);
              const float z = HZ ? F::value(zc[u][q][h]) : 0.0f;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float d = HZ ? fmaf(-z, xsum[t][h][j], c[j]) : c[j];
                total[q][t][j] = fmaf(s, d, total[q][t][j]);
              }
            }
        }
      }
    }
#pragma unroll
    for (int q = 0; q < NR; ++q)
#pragma unroll
      for (int t = 0; t < TT; ++t) red[(wave * NR * TT + q * TT + t) * 64 + lane] = total[q][t];
    __syncthreads();
    // output tile o: summed over the waves and stored by wave o % waves
    for (int o = wave; o < NO * TT; o += waves) {
      f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f}, up = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int p = 0; p < waves; ++p) {
        v += red[(p * NR * TT + o) * 64 + lane];
        if (GATED) up += red[(p * NR * TT + NO * TT + o) * 64 + lane];
      }
      const int n = n0 + 16 * (o / TT) + l;
      if (n >= NH) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const long r = r0 + 16 * (o % TT) + 4 * g + j;
        if (r >= r_end) continue;
        const float y = GATED ? silu_mul(v[j], up[j]) : v[j];
        if (otype == MOE_T_F32) ((float*)a.out)[r * a.ldo + n] = y;
        else store_out((uint16_t*)a.out + r * a.ldo + n, y, std::integral_constant<int, XT>());
      }
    }
    __syncthreads();
  }
}

int bad(int code, const char* msg) {
  moe_set_thread_error(msg);
  return code;
}

template <int XT, int GM, int NR, int TT, bool GATED, bool HZ>
void launch(const W4Args& a, int otype, hipStream_t s) {
  const int NO = GATED ? NR / 2 : NR;
  const int NH = GATED ? a.N / 2 : a.N;
  const int steps = (a.K + 127) / 128, waves = steps < 4 ? steps : 4;
  const long ny = a.offsets ? (a.rows < a.E ? a.rows : a.E) : (a.rows + 16 * TT - 1) / (16 * TT);
  const dim3 grid((NH + 16 * NO - 1) / (16 * NO), (unsigned)ny);
  w4_kernel<XT, GM, NR, TT, GATED, HZ><<<grid, 64 * waves, (size_t)waves * NR * TT * 64 * 16, s>>>(a, otype);
}

template <int XT, int GM, bool HZ>
void choose(const W4Args& a, bool gated, int otype, hipStream_t s) {
  if (gated) {
    if (a.offsets || a.rows <= 16) launch<XT, GM, 2, 1, true, HZ>(a, otype, s);
    else if (a.rows <= 32) launch<XT, GM, 2, 2, true, HZ>(a, otype, s);
    else launch<XT, GM, 4, 4, true, HZ>(a, otype, s);
  } else {
    if (a.offsets || a.rows <= 16) launch<XT, GM, 1, 1, false, HZ>(a, otype, s);
    else if (a.rows <= 32) launch<XT, GM, 2, 2, false, HZ>(a, otype, s);
    else launch<XT, GM, 4, 4, false, HZ>(a, otype, s);
  }
}

template <int XT>
void choose_group(const W4Args& a, bool gated, int otype, hipStream_t s) {
  const int gm = a.G % 128 == 0 ? 128 : a.G;
  if (a.zeros) {
    if (gm == 128) choose<XT, 128, true>(a, gated, otype, s);
    else if (gm == 64) choose<XT, 64, true>(a, gated, otype, s);
    else choose<XT, 32, true>(a, gated, otype, s);
  } else {
    if (gm == 128) choose<XT, 128, false>(a, gated, otype, s);
    else if (gm == 64) choose<XT, 64, false>(a, gated, otype, s);
    else choose<XT, 32, false>(a, gated, otype, s);
  }
}

}  // namespace

extern "C" int moe_w4_matmul(int xtype, const void* x, int64_t ldx, int64_t x_rows, const int32_t* row_map,
                             int map_div, const int32_t* offsets, const int32_t* counts, int E, int64_t rows,
                             const uint8_t* codes, int stype, const void* scales, const void* zeros, int N, int K,
                             int group, int gated, int otype, void* out, int64_t ldo, void* stream) {
  if (xtype != MOE_T_BF16 && xtype != MOE_T_F16) return bad(MOE_E_INVAL, "x is bf16 or fp16");
  if (stype != MOE_T_BF16 && stype != MOE_T_F16) return bad(MOE_E_INVAL, "scales are bf16 or fp16");
  if (otype != xtype && otype != MOE_T_F32) return bad(MOE_E_INVAL, "out has x's type or is fp32");
  if (N < 1 || K < 1 || (gated && N % 2)) return bad(MOE_E_INVAL, "need N >= 1 (even when gated) and K >= 1");
  if (group != 32 && group != 64 && (group < 128 || group % 128))
    return bad(MOE_E_INVAL, "group: 32, 64 or a multiple of 128");
  if (K % group) return bad(MOE_E_INVAL, "K is a multiple of the group");
  if (rows < 0 || rows > 0x7fffffffLL || x_rows < 0) return bad(MOE_E_INVAL, "rows outside [0, 2^31)");
  if (E < 1 || E > 1024) return bad(MOE_E_INVAL, "need 1 <= E <= 1024");
  if (!offsets && (E != 1 || counts)) return bad(MOE_E_INVAL, "without offsets: one matrix and no counts");
  if (row_map && map_div < 1) return bad(MOE_E_INVAL, "need map_div >= 1");
  if (!row_map && x_rows < rows) return bad(MOE_E_INVAL, "x has fewer rows than out");
  if (ldx < K || ldx % 8) return bad(MOE_E_INVAL, "x's row stride: at least K and a multiple of 8");
  if (ldo < (gated ? N / 2 : N)) return bad(MOE_E_INVAL, "out's row stride smaller than its width");
  if (rows == 0) return MOE_OK;
  if ((x_rows && !x) || !codes || !scales || !out) return bad(MOE_E_INVAL, "null argument");
  if (((uintptr_t)x | (uintptr_t)codes) % 16) return bad(MOE_E_INVAL, "x and codes start on 16 bytes");
  W4Args a{(const uint16_t*)x, ldx, x_rows, row_map, map_div, offsets, counts, E, rows, codes, (const uint16_t*)scales,
           (const uint16_t*)zeros, N, K, group, stype == MOE_T_F16, out, ldo};
  if (!offsets && (rows + 15) / 16 > 65535) return bad(MOE_E_UNSUPPORTED, "more than 1048560 rows");
  if (xtype == MOE_T_BF16) choose_group<MOE_T_BF16>(a, gated != 0, otype, (hipStream_t)stream);
  else choose_group<MOE_T_F16>(a, gated != 0, otype, (hipStream_t)stream);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? MOE_OK : bad(MOE_E_HIP, hipGetErrorString(e));
}
