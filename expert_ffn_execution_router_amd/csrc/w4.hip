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
#include "fwd_ws.h"
#include "moe.h"
#include "route_dev.h"
#include "spans.h"

#include <algorithm>

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
  int N, K, NG;                // NG groups per weight row
  uint32_t per_group;          // 2^31 over the runs of 32, 64 or 128 inputs in a group, rounded up
  void* out;
  long ldo;
};

// Workgroup barrier after LDS writes that leaves global loads in flight.
DEV void barrier_lds() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

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
// integers, the even inputs before the odd ones (input order costs two
// instructions more; the x rows are put in this order once instead).
template <int XT>
DEV typename Frag<XT>::type codes8(uint32_t w) {
  const uint32_t a = w & 0x0F0F0F0Fu, b = (w >> 4) & 0x0F0F0F0Fu;
  const i32x4_t v = {(int)Frag<XT>::lo(a), (int)Frag<XT>::hi(a), (int)Frag<XT>::lo(b), (int)Frag<XT>::hi(b)};
  return __builtin_bit_cast(typename Frag<XT>::type, v);
}

// 8 inputs with the even ones first.
DEV i32x4_t even_first(i32x4_t x) {
  const auto pick = [](int lo, int hi, uint32_t sel) { return (int)__builtin_amdgcn_perm((uint32_t)hi, (uint32_t)lo, sel); };
  return i32x4_t{pick(x[0], x[1], 0x05040100u), pick(x[2], x[3], 0x05040100u), pick(x[0], x[1], 0x07060302u),
                 pick(x[2], x[3], 0x07060302u)};
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

// The want-th block of up to 16 rows (of one expert) in expert order, and its
// rows [at, end); false if there are fewer.  Every wave finds it for itself:
// four runs of 64 experts are loaded together, a wave scan counts their
// blocks.
DEV bool find_rows(const W4Args& a, int want, size_t& e, long& at, long& end) {
  constexpr int R = 16;
  const int lane = threadIdx.x & 63;
  for (int e0 = 0; e0 < a.E; e0 += 256) {
    // loads without branches, so that they are in flight together
    int o[4], c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int ee = min(e0 + 64 * i + lane, a.E - 1);
      o[i] = a.offsets[ee];
      c[i] = a.counts ? a.counts[ee] : a.offsets[ee + 1];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (!a.counts) c[i] -= o[i];
      if (e0 + 64 * i + lane >= a.E) c[i] = 0;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int mine = c[i] > 0 ? (c[i] + R - 1) / R : 0;
      const int sum = wave_incl_sum(mine);
      const int here = __builtin_amdgcn_readlane(sum, 63);
      if (want >= here) {
        want -= here;
        continue;
      }
      const int b = __builtin_ctzll(__builtin_amdgcn_ballot_w64(sum > want));
      e = e0 + 64 * i + b;
      const long off = __builtin_amdgcn_readlane(o[i], b);
      end = off + __builtin_amdgcn_readlane(c[i], b);
      at = off + (long)R * (want - __builtin_amdgcn_readlane(sum - mine, b));
      if (end > at + R) end = at + R;
      if (end > a.rows) end = a.rows;
      if (off < 0 || at > a.rows) at = end = 0;  // offsets that are none: no rows
      return true;
    }
  }
  return false;
}

// Bound on the blocks of up to 16 rows for any grouping of a call's rows.
long row_blocks(const W4Args& a) {
  if (!a.offsets) return (a.rows + 15) / 16;
  const long experts = a.rows < a.E ? a.rows : a.E;
  return experts + (a.rows - experts) / 16;
}

// What rows without an x row read.
constexpr int MAX_K = 32768;
alignas(16) __device__ uint16_t w4_zeros[MAX_K];

// The x row that grouped row r reads, zeros if there is none; r not below end
// reads the last row's (for result rows that are not stored).
DEV const uint16_t* x_row(const W4Args& a, long r, long end) {
  if (r >= end) r = end > 0 ? end - 1 : 0;
  long src = r;
  if (a.row_map) {
    const int m = a.row_map[r];
    src = m < 0 ? -1 : m / a.map_div;
  }
  return src >= 0 && src < a.xrows ? a.x + src * a.ldx : w4_zeros;
}

// Sum over the PER fragments of a group of x times the value that cst holds
// twice, the same in every column.
template <int XT, int PER>
DEV f32x4_t group_xsum(const typename Frag<XT>::type* x, int cst) {
  typedef typename Frag<XT>::type frag;
  const frag cf = __builtin_bit_cast(frag, (i32x4_t){cst, cst, cst, cst});
  f32x4_t c = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < PER; ++i) c = Frag<XT>::mfma(x[i], cf, c);
  return c;
}

// First input of fragment i of a step for lane row g.
template <int GM>
DEV constexpr int frag_k(int g, int i) { return GM == 128 ? 32 * g + 8 * i : 32 * i + 8 * g; }

// One word of each of the four lane rows, for all lane rows.
DEV void spread_rows(uint32_t v, uint32_t (&o)[4]) {
  const auto a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  const auto b = __builtin_amdgcn_permlane16_swap(a[0], a[0], false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[1], a[1], false, false);
  o[0] = b[0];
  o[1] = b[1];
  o[2] = c[0];
  o[3] = c[1];
}

// A workgroup takes 16 x rows of one matrix and `per` groups of NR tiles of 16
// weight rows (gated: NR / 2 gate tiles and the matching up tiles).  Its waves
// split the inputs: each keeps its S steps of 128 inputs of the x rows in
// registers, with their sums per group, and multiplies one tile group after
// the other, all of whose codes it loads together; the loads of the next group
// run while the waves' sums of this one are added, through LDS and in wave
// order, and stored.  Loads have no branches, so that a wait counts exactly
// the loads behind it: what lies past the inputs repeats the last codes (their
// x are zeros), what lies past the matrix its last rows.
//
// In a step lane (g, l) of a wave (g = lane / 16) holds 32 codes (16 bytes) of
// weight row l at inputs 32 g ..; as operand fragment i they are inputs
// 32 g + 8 i .. for groups of 128 and more (the group spans the step, so the
// order of its inputs is free as long as x is read alike), and for smaller
// groups the words are exchanged between the lane rows so that fragment i
// holds inputs 32 i + 8 g ..: one fragment is then one run of 32 inputs.  The
// group values of two steps and two tiles come in one load, lane (g, l)
// reading step g % 2 of tile g / 2 for row l, so every loaded byte is a
// different one; the lane rows then hand them to each other.
//
// Codes are loaded without the nontemporal hint: a load takes half of a
// 128-byte line of each row, the load of the next step the other half.  With
// weights that rotate past the last-level cache, without against with the
// hint: 60 against 73 us for 64 rows, 6144 -> 2 x 6144, 46 against 51 us for
// 64 tokens x 8 of 128 experts, 2048 -> 2 x 768.
//
// What bounds it with few rows is vector work and the latency of the codes: a
// wave spends 39 vector instructions per KB of codes (63 with groups of 64 and
// zeros) besides the matrix ones, and a tile group's loads are in flight only
// while the last one's sums are added.  64 tokens x 8 of 128, 2048 -> 2 x 768
// and 32 tokens x 6 of 256, 2048 -> 4096, groups of 64 with zeros, both stream
// 3.7 TB/s.  Past 16 rows the codes are converted again for every 16, and past
// 2048 inputs x, twice the codes' bytes, is read again for every tile group.
constexpr int MAX_WAVES = 8;

template <int XT, int ST, int GM, int S, bool LONG, bool GATED, bool HZ>
__global__ void __launch_bounds__(64 * MAX_WAVES, S <= 2 ? 4 : 2)
w4_kernel(W4Args a, int otype, int blocks, int per, int passes) {
  typedef typename Frag<XT>::type frag;
  constexpr int SUB = 128 / GM, PER = 4 / SUB, NW = (SUB + 1) / 2, NR = 2, NO = GATED ? NR / 2 : NR;
  constexpr bool KEEP = S * SUB <= 2 && !LONG;            // sums of x kept, else taken again for each group
  constexpr bool TIGHT = SUB == 4 || S > 2 || (SUB == 2 && HZ);
  extern __shared__ float red[];                 // [waves][NR][row quads][64]
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int waves = blockDim.x >> 6, g = lane >> 4, l = lane & 15;
  const int NH = GATED ? a.N / 2 : a.N, tiles = (NH + 15) / 16, K2 = a.K / 2;
  const int t0 = blockIdx.x * per * NO, t_end = min(tiles, t0 + per * NO);
  // the lane's place in its steps of pass p: codes, and group values of a
  // pair of steps
  uint32_t off[S];
  int grp[S / 2];
  const auto place = [&](int p) {
#pragma unroll
    for (int s = 0; s < S; ++s) off[s] = (uint32_t)min(64 * ((p * waves + wave) * S + s) + 16 * g, K2 - 16);
#pragma unroll
    for (int s = 0; s < S / 2; ++s) {
      const int st = (p * waves + wave) * S + 2 * s + (g & 1);
      grp[s] = SUB > 1 ? st * SUB : (int)min((uint32_t)(((uint64_t)(uint32_t)st * a.per_group) >> 31), (uint32_t)a.NG - 1);
    }
  };
  place(0);
  for (int blk = blockIdx.y; blk < blocks; blk += gridDim.y) {
    long r0, r_end;
    size_t e = 0;
    if (a.offsets) {
      if (!find_rows(a, blk, e, r0, r_end)) return;             // past the last block
    } else {
      r0 = (long)blk * 16;
      r_end = r0 + 16 < a.rows ? r0 + 16 : a.rows;
    }
    const uint8_t* const wbase = a.codes + e * a.N * K2;
    const size_t gbase = e * a.N * a.NG;
    const int glast = (int)min((long)a.E * a.N * a.NG - SUB - (long)gbase, (long)0x7fffffff);
    int cst = HZ ? Frag<XT>::ONE : Frag<XT>::MINUS8;
    i32x4_t w[S][NR];
    uint64_t sc[S / 2][NR / 2], z[S / 2][NR / 2];
    const auto load = [&](int tile0) {
      int row[NR];                               // first row of the tile, and the lane's row in it
      uint32_t lr[NR];
#pragma unroll
      for (int q = 0; q < NR; ++q) {
        const int tile = min(tile0 + q % NO, tiles - 1);
        row[q] = (q / NO) * NH + 16 * tile;
        lr[q] = (uint32_t)min(l, NH - 1 - 16 * tile);
      }
#pragma unroll
      for (int q = 0; q < NR; ++q)
#pragma unroll
        for (int s = 0; s < S; ++s) w[s][q] = ld16(wbase + (size_t)row[q] * K2 + (lr[q] * K2 + off[s]));
#pragma unroll
      for (int p = 0; p < NR / 2; ++p)
#pragma unroll
        for (int s = 0; s < S / 2; ++s) {
          const int r = g >= 2 ? row[2 * p + 1] + (int)lr[2 * p + 1] : row[2 * p] + (int)lr[2 * p];
          const int want = r * a.NG + grp[s];
          // read from an earlier place where it would pass the end of all values
          const int from = SUB > 1 ? min(want, glast) : want, sh = SUB > 1 ? min(16 * (want - from), 63) : 0;
          uint64_t v = 0;
          __builtin_memcpy(&v, a.scales + gbase + from, 2 * SUB);
          sc[s][p] = v >> sh;
          if (HZ) {
            uint64_t u = 0;
            __builtin_memcpy(&u, a.zeros + gbase + from, 2 * SUB);
            z[s][p] = u >> sh;
          }
        }
    };
    int first = t0;
    asm volatile("" : "+s"(first));             // its addresses are not kept over the blocks
    if (LONG) place(0);
    load(first);
    frag x[S][4];
    f32x4_t kept[KEEP ? S : 1][SUB];
    const uint16_t* xr = x_row(a, r0 + l, r_end);
    const auto load_x = [&](int p) {
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int k = 128 * ((p * waves + wave) * S + s) + frag_k<GM>(g, i);
          x[s][i] = __builtin_bit_cast(frag, even_first(ld16(k < a.K ? xr + k : w4_zeros)));
        }
    };
    if (!LONG) load_x(0);
    if (KEEP)
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int h = 0; h < SUB; ++h) kept[KEEP ? s : 0][h] = group_xsum<XT, PER>(x[s] + h * PER, cst);
    // row quads that are stored, in LDS a power of two of them
    const int rows = (int)(r_end - r0), ql = rows > 8 ? 2 : (rows > 4 ? 1 : 0);
    f32x4_t total[NR];
    const auto multiply = [&]() {
      if (!KEEP) asm volatile("" : "+v"(cst));     // the sums of x are not hoisted out of the loop
#pragma unroll
      for (int s2 = 0; s2 < S / 2; ++s2) {
        uint32_t sv[NR / 2][NW][4], zv[NR / 2][NW][4];
#pragma unroll
        for (int p = 0; p < NR / 2; ++p)
#pragma unroll
          for (int i = 0; i < NW; ++i) {
            spread_rows((uint32_t)(sc[s2][p] >> (32 * i)), sv[p][i]);
            if (HZ) spread_rows((uint32_t)(z[s2][p] >> (32 * i)), zv[p][i]);
          }
#pragma unroll
        for (int s1 = 0; s1 < 2; ++s1) {
          const int s = 2 * s2 + s1;
          i32x4_t c4[NR];
#pragma unroll
          for (int q = 0; q < NR; ++q) {
            c4[q] = w[s][q];
            if (GM < 128) transpose_rows(c4[q]);
          }
#pragma unroll
          for (int h = 0; h < SUB; ++h) {
            // the group's codes are not used before the last group's sums are
            // done: all groups' results at once do not fit the registers
            if (TIGHT)
#pragma unroll
              for (int q = 0; q < NR; ++q) asm volatile("" : "+v"(total[q]), "+v"(c4[q]));
            const f32x4_t xsum = KEEP ? kept[KEEP ? s : 0][h] : group_xsum<XT, PER>(x[s] + h * PER, cst);
#pragma unroll
            for (int q = 0; q < NR; ++q) {
              const int from = s1 + 2 * (q & 1);                // the lane row that loaded it
              const float sf = Frag<ST>::value((uint16_t)(sv[q / 2][h / 2][from] >> (16 * (h & 1))));
              const float zf = HZ ? Frag<XT>::value((uint16_t)(zv[q / 2][h / 2][from] >> (16 * (h & 1)))) : 0.0f;
              f32x4_t c = HZ ? f32x4_t{0.0f, 0.0f, 0.0f, 0.0f} : xsum;
#pragma unroll
              for (int j = h * PER; j < (h + 1) * PER; ++j)
                c = Frag<XT>::mfma(x[s][j], codes8<XT>((uint32_t)c4[q][j]), c);
#pragma unroll
              for (int j = 0; j < 4; ++j) total[q][j] = fmaf(sf, HZ ? fmaf(-zf, xsum[j], c[j]) : c[j], total[q][j]);
            }
          }
        }
      }
    };
    for (int tile0 = t0;;) {
#pragma unroll
      for (int q = 0; q < NR; ++q) total[q] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
      if (!LONG) {
        multiply();
      } else {
        for (int p = 0;;) {
          load_x(p);
          multiply();
          if (++p == passes) break;
          place(p);
          load(tile0);
        }
      }
      const int tile1 = tile0 + NO;
      const bool more = tile1 < t_end;
      if (more) {
        if (LONG) place(0);
        load(tile1);
      }
      if (4 * g < rows)
#pragma unroll
        for (int q = 0; q < NR; ++q) *(f32x4_t*)(red + (((wave * NR + q) << ql) + g) * 64 + 4 * l) = total[q];
      barrier_lds();
      // a share: one row quad of one tile, a value a lane
      for (int f = wave; f < NO << ql; f += waves) {
        const int o = f >> ql, qd = f & ((1 << ql) - 1);
        const float* p = red + f * 64 + lane;
        float v = 0.0f, up = 0.0f;
#pragma unroll
        for (int k = 0; k < MAX_WAVES; ++k) {
          const int at = (min(k, waves - 1) * NR << ql) * 64;
          const float m = p[at], n = GATED ? p[at + (NO << ql) * 64] : 0.0f;
          v += k < waves ? m : 0.0f;
          if (GATED) up += k < waves ? n : 0.0f;
        }
        if (GATED) v = silu_mul(v, up);
        const int r = 4 * qd + (lane & 3), col = 16 * (tile0 + o) + (lane >> 2);
        if (r < rows && col < NH) {
          const long at = (r0 + r) * a.ldo + col;
          if (otype == MOE_T_F32) ((float*)a.out)[at] = v;
          else store_out((uint16_t*)a.out + at, v, std::integral_constant<int, XT>());
        }
      }
      if (!more) break;
      barrier_lds();                                            // red is free
      tile0 = tile1;
    }
    if (blk + gridDim.y < blocks) barrier_lds();
  }
}

int bad(int code, const char* msg) {
  moe_set_thread_error(msg);
  return code;
}

template <int XT, int ST, int GM, int S, bool LONG, bool GATED, bool HZ>
void launch(const W4Args& a, int otype, hipStream_t s) {
  // Tile groups per workgroup, so that about WGS workgroups share the list (two
  // are resident on each of 256 CUs): the x rows are read once for them and
  // their loads overlap the sums of the one before.  At most PER of them, as
  // grouped rows have a bound on their blocks only and fewer may be there.
  constexpr long WGS = 1024, PER = 8;
  constexpr int NO = GATED ? 1 : 2;
  const int steps = (a.K + 127) / 128, passes = LONG ? (steps + S * MAX_WAVES - 1) / (S * MAX_WAVES) : 1;
  const int waves = (steps + S * passes - 1) / (S * passes);
  const long groups = (((GATED ? a.N / 2 : a.N) + 15) / 16 + NO - 1) / NO, blocks = row_blocks(a);
  const long per = std::min(std::max(groups * blocks / WGS, 1L), PER), gx = (groups + per - 1) / per;
  // the grid stops at 4 WGS workgroups, which take the row blocks beyond in turn
  const long ny = std::min(std::min(blocks, std::max(4 * WGS / gx, 1L)), 65535L);
  w4_kernel<XT, ST, GM, S, LONG, GATED, HZ><<<dim3((unsigned)gx, (unsigned)ny), 64 * waves, (size_t)waves * 2048, s>>>(
      a, otype, (int)blocks, (int)per, passes);
}

// Two steps of inputs per wave (their group values come in pairs) hold rows of
// up to 2048; longer rows are taken in passes, the x rows read again for each
// tile pair.  Rows of up to 4096 can be held with four steps, on half the
// waves: many tile pairs win that back by not reading x again.  Held against
// passes in us, weights rotating past the last-level cache, groups of 128:
//   tile pairs       512      1024       2048       4096       8192
//   4096 inputs  20 / 18   35 / 28   48 /  52   70 /  98  116 / 191
//   2176 inputs  15 / 11   25 / 22   34 /  36   51 /  66   86 / 128
//   64 experts, 32 tokens x 4, 4096 rows (8704 pairs), 4096 inputs: 86 / 110
// Groups of 32 and 64 cross later and less (4096 inputs, groups of 32: 58 / 53
// at 2048, 90 / 99 at 4096, 158 / 191 at 8192), hence 4096.  With few rows per
// expert they go either way past it: 128 experts, 64 tokens x 8, 2176 inputs,
// groups of 64: 2048 weight rows 111 / 128, with zeros 150 / 145, 4096 with
// zeros 272 / 235.
template <int XT, int ST, int GM, bool GATED, bool HZ>
void choose(const W4Args& a, int otype, hipStream_t s) {
  const int steps = (a.K + 127) / 128;
  const long pairs = (((GATED ? a.N / 2 : a.N) + 15) / 16 + (GATED ? 0 : 1)) / (GATED ? 1 : 2) * row_blocks(a);
  if (steps <= 2 * MAX_WAVES) launch<XT, ST, GM, 2, false, GATED, HZ>(a, otype, s);
  else if (steps <= 4 * MAX_WAVES && pairs >= 4096) launch<XT, ST, GM, 4, false, GATED, HZ>(a, otype, s);
  else launch<XT, ST, GM, 2, true, GATED, HZ>(a, otype, s);
}

template <int XT, int ST, bool GATED, bool HZ>
void choose_group(const W4Args& a, int otype, hipStream_t s) {
  const int group = a.NG == 1 ? 128 : a.K / a.NG;           // with one group its inputs past K are zeros
  if (group == 32) choose<XT, ST, 32, GATED, HZ>(a, otype, s);
  else if (group == 64) choose<XT, ST, 64, GATED, HZ>(a, otype, s);
  else choose<XT, ST, 128, GATED, HZ>(a, otype, s);
}

template <int XT, int ST>
void choose_form(const W4Args& a, bool gated, int otype, hipStream_t s) {
  if (gated) a.zeros ? choose_group<XT, ST, true, true>(a, otype, s) : choose_group<XT, ST, true, false>(a, otype, s);
  else a.zeros ? choose_group<XT, ST, false, true>(a, otype, s) : choose_group<XT, ST, false, false>(a, otype, s);
}

}  // namespace

extern "C" int moe_w4_matmul(int xtype, const void* x, int64_t ldx, int64_t x_rows, const int32_t* row_map,
                             int64_t map_div, const int32_t* offsets, const int32_t* counts, int64_t E, int64_t rows,
                             const uint8_t* codes, int stype, const void* scales, const void* zeros, int64_t N,
                             int64_t K, int64_t group, int gated, int otype, void* out, int64_t ldo, void* stream) {
  if (xtype != MOE_T_BF16 && xtype != MOE_T_F16) return bad(MOE_E_INVAL, "x is bf16 or fp16");
  if (stype != MOE_T_BF16 && stype != MOE_T_F16) return bad(MOE_E_INVAL, "scales are bf16 or fp16");
  if (otype != xtype && otype != MOE_T_F32) return bad(MOE_E_INVAL, "out has x's type or is fp32");
  if (N < 1 || K < 1 || (gated && N % 2)) return bad(MOE_E_INVAL, "need N >= 1 (even when gated) and K >= 1");
  if (group != 32 && group != 64 && (group < 128 || group % 128))
    return bad(MOE_E_INVAL, "group: 32, 64 or a multiple of 128");
  if (K % group) return bad(MOE_E_INVAL, "K is a multiple of the group");
  if (K > MAX_K) return bad(MOE_E_UNSUPPORTED, "K over 32768");
  if (rows < 0 || rows > 0x7fffffffLL || x_rows < 0) return bad(MOE_E_INVAL, "rows outside [0, 2^31)");
  if (E < 1 || E > 1024) return bad(MOE_E_INVAL, "need 1 <= E <= 1024");
  if (N > 1 << 30 || N * (K / group) > 1 << 30) return bad(MOE_E_UNSUPPORTED, "more than 2^30 groups in a matrix");
  // the group values of a step come in one load: 4 of them, 2 for groups of 64
  // (K holds two such groups at least), 1 otherwise
  if (group == 32 && K != group && E * N * (K / group) < 4)
    return bad(MOE_E_UNSUPPORTED, "fewer than 4 groups of 32 in all");
  if (!offsets && (E != 1 || counts)) return bad(MOE_E_INVAL, "without offsets: one matrix and no counts");
  if (row_map && (map_div < 1 || map_div > 0x7fffffff)) return bad(MOE_E_INVAL, "need 1 <= map_div < 2^31");
  if (!row_map && x_rows < rows) return bad(MOE_E_INVAL, "x has fewer rows than out");
  if (ldx < K || ldx % 8) return bad(MOE_E_INVAL, "x's row stride: at least K and a multiple of 8");
  if (ldo < (gated ? N / 2 : N)) return bad(MOE_E_INVAL, "out's row stride smaller than its width");
  if (rows == 0) return MOE_OK;
  if ((x_rows && !x) || !codes || !scales || !out) return bad(MOE_E_INVAL, "null argument");
  if (((uintptr_t)x | (uintptr_t)codes) % 16) return bad(MOE_E_INVAL, "x and codes start on 16 bytes");
  const int64_t values = E * N * (K / group) * 2;
  if (outputs_shared({row_span(out, rows, gated ? N / 2 : N, ldo, otype == MOE_T_F32 ? 4 : 2)},
                     {row_span(x, x_rows, K, ldx, 2), span(row_map, rows * 4), span(offsets, (E + 1) * 4),
                      span(counts, E * 4), span(codes, E * N * (K / 2)), span(scales, values), span(zeros, values)}))
    return bad(MOE_E_INVAL, "out shares memory with an input");
  // sizes came in 64 bits, so that none is cut before its check; they fit an int now
  W4Args a{(const uint16_t*)x, ldx, x_rows, row_map, (int)map_div, offsets, counts, (int)E, rows, codes,
           (const uint16_t*)scales, (const uint16_t*)zeros, (int)N, (int)K, (int)(K / group), 0, out, ldo};
  const uint32_t runs = group < 128 ? 1 : (uint32_t)group / 128;      // a step never passes a group of more than 128
  a.per_group = ((1u << 31) + runs - 1) / runs;
  const hipStream_t s = (hipStream_t)stream;
  constexpr int BF = MOE_T_BF16, HF = MOE_T_F16;
  if (xtype == BF) stype == BF ? choose_form<BF, BF>(a, gated, otype, s) : choose_form<BF, HF>(a, gated, otype, s);
  else stype == BF ? choose_form<HF, BF>(a, gated, otype, s) : choose_form<HF, HF>(a, gated, otype, s);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? MOE_OK : bad(MOE_E_HIP, hipGetErrorString(e));
}
