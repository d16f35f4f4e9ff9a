// Products of E4M3 codes with a scale for each 128 of the summed axis.
//
//   rows:   out[r, n] = sum_g sa[g, r] sw[n / 128, g] sum_{k in group g} a[r, k] w[n, k]
//   depth:  dw[n, k]  = sum_G sdy[G, n] sx[G, k] sum_{t in group G} dy[t, n] x[t, k]
//
// In both a row operand P (a, dy transposed) with a scale per row and group
// meets a column operand Q (w, x transposed) with a scale per block of 128 or
// per column and group; both are summed along their contiguous axis.
#include <cmath>

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
  int split;                   // depth: parts of the summed axis, out [E][split][R][ldo]
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

// ---------------------------------------------------------------------------
// few rows
// ---------------------------------------------------------------------------
// A workgroup takes 16 columns of Q and up to 16 RT rows of P; its 8 waves
// share out the groups, read both operands straight into registers (a lane's 16
// bytes twice per group: whole 128-byte lines of a row) and join their sums in
// LDS.  The matrix instruction's columns are rows of P and its rows columns of
// Q, so a lane ends with four neighbours of one row.  The 8-bit instruction's
// sum of neighbouring products keeps fewer bits than fp32, and here the
// weights' bytes are the bound, so the codes are multiplied as fp16, which is
// exact.  32 rows, 4096 x 4096: 9.8 us alone (17 MB, 1.8 TB/s: a launch, the
// loads' latency twice and the join), 34 with the weights through LDS.
constexpr int STREAM_WAVES = 8;

template <int RT>
__global__ void __launch_bounds__(64 * STREAM_WAVES, 2)
stream_kernel(MmArgs a, int row_blocks) {
  constexpr int U = RT == 4 ? 2 : 4;             // groups loaded together
  __shared__ __align__(16) f32x4_t red[STREAM_WAVES][RT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, lr = lane & 15, lg = lane >> 4;
  const int64_t c0 = (int64_t)blockIdx.x * 16;
  const int G = a.groups;
  for (int blk = blockIdx.y; blk < row_blocks; blk += gridDim.y) {
    RowBlock b{0, (int64_t)blk * 16 * RT, min((int64_t)(blk + 1) * 16 * RT, a.R)};
    if (a.offsets && !find_block<16 * RT>(a.offsets, a.counts, a.E, a.R, blk, b)) return;
    const uint8_t* q = a.q + ((int64_t)b.e * a.C + min(c0 + lr, a.C - 1)) * a.ldk + 16 * lg;
    const float* sq = a.sq + ((int64_t)b.e * ((a.C + 127) / 128) + c0 / 128) * G;
    const uint8_t* p[RT];
    const float* sp[RT];
#pragma unroll
    for (int j = 0; j < RT; ++j) {               // past the last row it again, not stored
      const int64_t r = min(b.at + 16 * j + lr, b.end - 1);
      p[j] = a.p + r * a.ldk + 16 * lg;
      sp[j] = a.sp + r;
    }
    f32x4_t acc[RT] = {};
    i32x4_t qn[U][2];
    const auto load = [&](int g0) {              // past the last group it again, unused
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t g = min(g0 + u * STREAM_WAVES, G - 1);
        qn[u][0] = ld16_nt(q + g * 128);
        qn[u][1] = ld16_nt(q + g * 128 + 64);
      }
    };
    load(wave);
    for (int g0 = wave; g0 < G; g0 += STREAM_WAVES * U) {
      i32x4_t qc[U][2], pv[U][RT][2];
      float s[U][RT];
      __builtin_memcpy(qc, qn, sizeof(qc));
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t g = min(g0 + u * STREAM_WAVES, G - 1);
        const float w = sq[g];
#pragma unroll
        for (int j = 0; j < RT; ++j) {
          pv[u][j][0] = ld16(p[j] + g * 128);
          pv[u][j][1] = ld16(p[j] + g * 128 + 64);
          s[u][j] = sp[j][g * a.R] * w;
        }
      }
      if (g0 + STREAM_WAVES * U < G) load(g0 + STREAM_WAVES * U);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (g0 + u * STREAM_WAVES >= G) break;
        f16x8_t m[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) m[h] = codes_f16(qc[u][h >> 1][2 * (h & 1)], qc[u][h >> 1][2 * (h & 1) + 1]);
#pragma unroll
        for (int j = 0; j < RT; ++j) {
          f32x4_t pr = {};
#pragma unroll
          for (int h = 0; h < 4; ++h)
            pr = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                m[h], codes_f16(pv[u][j][h >> 1][2 * (h & 1)], pv[u][j][h >> 1][2 * (h & 1) + 1]), pr, 0, 0, 0);
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[j][v] += pr[v] * s[u][j];
        }
      }
    }
#pragma unroll
    for (int j = 0; j < RT; ++j) red[wave][j][lane] = acc[j];
    __syncthreads();
    if (wave < RT) {                             // wave j sums the rows 16 j
      f32x4_t v = {};
#pragma unroll
      for (int w = 0; w < STREAM_WAVES; ++w) v += red[w][wave][lane];
      const int64_t r = b.at + 16 * wave + lr, c = c0 + 4 * lg;
      if (r < b.end)
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (c + u < a.C) store_value(a.out, r * a.ldo + c + u, a.otype, v[u]);
    }
    __syncthreads();                             // red is free
  }
}

// ---------------------------------------------------------------------------
// tiles
// ---------------------------------------------------------------------------
// A persistent workgroup of 8 waves (2 halves of the rows x 4 quarters of the
// columns) takes tiles of BM rows of P x BN columns of Q, one group of 128 of
// the summed axis after the other.  A group's codes come by direct
// global->LDS loads into one of NST stages: rows of 128 bytes whose 16-byte
// pieces are XORed with (row / 2) % 8, so that 16 rows read at one place cover
// all banks; the scales behind them.  Every wave issues the same number of
// loads for a group, so the wait for a stage leaves exactly the later ones
// outstanding.  Rows past an edge repeat the last one and are not stored.
// 8192 x 4096 x 4096 in 167 us (1.6 PFLOP/s): each 128 of the summed axis costs
// a fused multiply-add per result beside its matrix instruction.  The sums take
// half of the 256 x 256 tile's registers and the operands the rest but for one
// or two results, so a matrix instruction is waited for in full by its
// multiply-adds, and each read of P too; deeper stages, wave priorities and
// fixed schedules changed nothing on so few registers.  The 8-bit instruction
// adds 8 neighbouring products at a time and drops of each what is under 2^-13
// of the largest one's power of two, toward zero: at most 2^-10 of that
// product, and of values alike 2^-16 of the sum of magnitudes.  That is a
// quarter of bf16's half step at worst where terms do not cancel, and a factor
// of two in time for many rows, so bf16 results take it; fp16 ones, whose step
// it could pass, and fp32 ones (EXACT) do not.  Experts of 4096 tokens on 4.6
// GB of weights in 1000 us (4.6 TB/s). Gradients of 128 experts, 1536 x 2048,
// in 850 us (1.6 GB written; taken apart, the stores alone took 280, loads and
// products 600, loads and stores 535: the memory path of a CU and its vector
// work are shared by all three): the codes are converted to fp16, as fp32
// results need every bit.
template <bool DEPTH, bool EXACT, int SUB, int NS>
struct Tile {
  static constexpr int BM = 32 * SUB, BN = 64 * NS;
  static constexpr int LOADS = (BM + BN) / 64;             // 1 KiB blocks of 8 rows for each wave
  static constexpr int P_OFF = 0, Q_OFF = BM * 128;
  static constexpr int SP_OFF = Q_OFF + BN * 128;          // scales: 64 floats a wave, 8 waves
  static constexpr int STAGE = SP_OFF + 8 * 256;
  static constexpr int NST = (160 * 1024 - 4352) / STAGE < 6 ? (160 * 1024 - 4352) / STAGE : 6;
  static constexpr int LDS = NST * STAGE;
};
constexpr int MAX_E = 1024;

DEV int swizzled(int row, int piece) { return row * 128 + ((piece ^ ((row >> 1) & 7)) << 4); }
DEV i32x4_t lds16(const uint8_t* p) { return *(const i32x4_t*)p; }
DEV void dma16(const void* src, lds_u8_t* dst) {
  __builtin_amdgcn_global_load_lds((gbl_void_t*)src, (lds_void_t*)dst, 16, 0, 0);
}
DEV void dma4(const void* src, lds_u8_t* dst) {
  __builtin_amdgcn_global_load_lds((gbl_void_t*)src, (lds_void_t*)dst, 4, 0, 0);
}

typedef float f32x4u_t __attribute__((ext_vector_type(4), aligned(4)));

// p[i] of an input, i the same in the wave, by a scalar load: a vector load's
// wait would be for every load and store in flight (gradients 862 -> 818 us).
DEV int constant(const int32_t* p, int i) {
  typedef const __attribute__((address_space(4))) int32_t* constant_t;
  return ((constant_t)(uintptr_t)p)[__builtin_amdgcn_readfirstlane(i)];
}

struct Item {
  int e, rows, cols, g0, g1;
  int64_t r0, c0;
};

template <bool DEPTH, bool EXACT, int SUB, int NS>
__global__ void __launch_bounds__(512, 2)
tile_kernel(MmArgs a) {
  using C = Tile<DEPTH, EXACT, SUB, NS>;
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ int pref[MAX_E + 1];                // m-tiles before each expert
  __shared__ int wave_tot[16];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int lr = lane & 15, lg = lane >> 4, wm = wave & 1, wn = wave >> 1;
  const int ntiles = (int)((a.C + C::BN - 1) / C::BN);
  const int dense_m = (int)((a.R + C::BM - 1) / C::BM);
  int nm_all = dense_m;
  if (!DEPTH && a.offsets) {
    int run[2], mine = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = 2 * tid + i;
      int c = 0;
      if (e < a.E) {
        const int64_t first = min(max((int64_t)a.offsets[e], (int64_t)0), a.R);
        const int64_t many = a.counts ? (int64_t)a.counts[e] : (int64_t)a.offsets[e + 1] - a.offsets[e];
        c = (int)((max(min(first + many, a.R) - first, (int64_t)0) + C::BM - 1) / C::BM);
      }
      run[i] = c;
      mine += c;
    }
    int sum = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(sum, d, 64);
      if (lane >= d) sum += v;
    }
    if (lane == 63) wave_tot[wave] = sum;
    __syncthreads();
    int before = sum - mine;
    nm_all = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i < wave) before += wave_tot[i];
      nm_all += wave_tot[i];
    }
    if (2 * tid <= a.E) pref[2 * tid] = before;
    if (2 * tid + 1 <= a.E) pref[2 * tid + 1] = before + run[0];
    if (tid == 511 && a.E == MAX_E) pref[MAX_E] = nm_all;
    __syncthreads();
  }
  const int nitems = nm_all * ntiles * (DEPTH ? a.E * a.split : 1);      // the host looked that it fits
  // each XCD deals its eighth of the list to its workgroups in turn
  constexpr int N_XCD = 8;
  const int xcd = blockIdx.x % N_XCD, per = (gridDim.x + N_XCD - 1 - xcd) / N_XCD;
  const int it1 = (int)((xcd + 1) * (int64_t)nitems / N_XCD);
  int it = (int)(xcd * (int64_t)nitems / N_XCD) + blockIdx.x / N_XCD;
  if (it >= it1) return;

  // The list goes expert by expert, four column tiles at a time over the
  // row tiles, so that workgroups side by side share both.
  const auto decode = [&](int i, Item& o) {
    int e = 0, nm = dense_m, first = 0, end = (int)a.R;
    unsigned q = i;
    o.g0 = 0;
    o.g1 = a.groups;
    if (DEPTH) {
      e = (int)((unsigned)i / (unsigned)(dense_m * ntiles));
      q = i - e * dense_m * ntiles;
      const int x = e / a.split, s = e - x * a.split;      // e: of the outputs
      if (a.offsets) {
        o.g0 = min(max(constant(a.offsets, x), 0) / 128, a.groups);
        o.g1 = max(min(max(constant(a.offsets, x + 1), 0) / 128, a.groups), o.g0);
      }
      const int64_t n = o.g1 - o.g0;
      o.g1 = o.g0 + (int)(n * (s + 1) / a.split);
      o.g0 += (int)(n * s / a.split);
    } else if (a.offsets) {
      const int m = (int)((unsigned)i / (unsigned)ntiles);
      int hi = a.E - 1;
      while (e < hi) {
        const int mid = (e + hi + 1) >> 1;
        if (pref[mid] <= m) e = mid; else hi = mid - 1;
      }
      nm = pref[e + 1] - pref[e];
      q = i - pref[e] * ntiles;
      const int64_t from = constant(a.offsets, e);
      first = (int)min(max(from, (int64_t)0), a.R);
      const int64_t many = a.counts ? (int64_t)constant(a.counts, e) : constant(a.offsets, e + 1) - from;
      end = (int)max(min(first + many, a.R), (int64_t)first);
    }
    nm = __builtin_amdgcn_readfirstlane(nm);
    q = __builtin_amdgcn_readfirstlane(q);
    first = __builtin_amdgcn_readfirstlane(first);
    end = __builtin_amdgcn_readfirstlane(end);
    const unsigned quad = q / (4u * nm), rest = q - quad * 4 * nm, wide = min(4, ntiles - 4 * (int)quad);
    const unsigned mt = rest / wide, nt = 4 * quad + rest - mt * wide;
    // equal tiles of the rows there are
    const unsigned step = (((unsigned)(end - first) + nm - 1) / (unsigned)nm + 15) & ~15u;
    const int64_t r0 = first + (int64_t)mt * step;
    o.e = __builtin_amdgcn_readfirstlane(e);
    o.rows = (int)max(min((int64_t)step, end - r0), (int64_t)0);
    const int64_t c0 = (int64_t)nt * C::BN;
    o.cols = (int)min((int64_t)C::BN, a.C - c0);
    o.g0 = __builtin_amdgcn_readfirstlane(o.g0);
    o.g1 = __builtin_amdgcn_readfirstlane(o.g1);
    o.r0 = r0;
    o.c0 = c0;
  };

  // ---- loads ----------------------------------------------------------------
  // Block b of the stage (8 rows): lane l brings the 16 bytes that belong at
  // piece l % 8 of row l / 8.
  const uint8_t* base[C::LOADS];
  const float* sbase = nullptr;
  int sstep = 0;
  const auto aim = [&](const Item& t) {
    const int last_r = max(t.rows - 1, 0), last_c = t.cols - 1;
    const uint8_t* p = a.p + t.r0 * a.ldk;
    const uint8_t* q = a.q + ((DEPTH ? 0 : t.e * a.C) + t.c0) * a.ldk;
#pragma unroll
    for (int i = 0; i < C::LOADS; ++i) {
      const int b = wave * C::LOADS + i;
      const bool isp = b < C::BM / 8;
      const int r = (isp ? b : b - C::BM / 8) * 8 + (lane >> 3), piece = (lane & 7) ^ ((r >> 1) & 7);
      base[i] = (isp ? p + (int64_t)min(r, last_r) * a.ldk : q + (int64_t)min(r, last_c) * a.ldk) + piece * 16;
    }
    // the wave's 64 scales: of P's rows, then of Q's
    constexpr int PW = (C::BM + 63) / 64;
    if (wave < PW) {
      sbase = a.sp + t.r0 + min(64 * wave + lane, last_r);
      sstep = (int)a.R;
    } else if (DEPTH) {
      sbase = a.sq + t.c0 + min(64 * min(wave - PW, C::BN / 64 - 1) + lane, last_c);
      sstep = (int)a.C;
    } else {                                     // block scales, BN / 128 of them (others repeat, unused)
      const int64_t cb = (a.C + 127) / 128;
      sbase = a.sq + (t.e * cb + min(t.c0 / 128 + (lane & 3), cb - 1)) * a.groups;
      sstep = 1;
    }
  };
  const auto issue = [&](int g, int stage) {
    lds_u8_t* sb = (lds_u8_t*)lds + stage * C::STAGE;
#pragma unroll
    for (int i = 0; i < C::LOADS; ++i) dma16(base[i] + (int64_t)g * 128, sb + (wave * C::LOADS + i) * 1024);
    dma4(sbase + (int64_t)g * sstep, sb + C::SP_OFF + wave * 256);
  };

  // ---- products -------------------------------------------------------------
  const int prow = 16 * SUB * wm + lr, qrow = 16 * NS * wn + lr;
  f32x4_t acc[NS][SUB];
  const auto clear = [&] {
#pragma unroll
    for (int i = 0; i < NS; ++i)
#pragma unroll
      for (int j = 0; j < SUB; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  };
  // the operand pieces: the fp8 instruction takes 32 neighbouring codes of a
  // lane group, the fp16 ones the same codes 8 at a time
  int p_rd[2], q_rd[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    p_rd[h] = C::P_OFF + swizzled(prow, 2 * lg + h);
    q_rd[h] = C::Q_OFF + swizzled(qrow, 2 * lg + h);
  }
  constexpr int PW = (C::BM + 63) / 64;
  const auto compute = [&](const uint8_t* sb) __attribute__((always_inline)) {
    const float* sps = (const float*)(sb + C::SP_OFF);
    const float* sqs = (const float*)(sb + C::SP_OFF + PW * 256);
    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
    if constexpr (!EXACT) {
      const float wsc = sqs[(16 * NS * wn) / 128];
      i32x8_t qv[NS];
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const i32x4_t lo = lds16(sb + q_rd[0] + i * 2048), hi = lds16(sb + q_rd[1] + i * 2048);
        qv[i] = i32x8_t{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      }
#pragma unroll
      for (int j = 0; j < SUB; ++j) {
        const i32x4_t lo = lds16(sb + p_rd[0] + j * 2048), hi = lds16(sb + p_rd[1] + j * 2048);
        const i32x8_t pv = i32x8_t{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        const float s = sps[prow + 16 * j] * wsc;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          const f32x4_t pr = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(qv[i], pv, zero, 0, 0, 0, 127, 0, 127);
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[i][j][v] += pr[v] * s;
        }
      }
    } else {
      f16x8_t qv[NS][4];
      f32x4_t qs[NS];
      const float wsc = DEPTH ? 1.0f : sqs[(16 * NS * wn) / 128];
#pragma unroll
      for (int i = 0; i < NS; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const i32x4_t w = lds16(sb + q_rd[h] + i * 2048);
          qv[i][2 * h] = codes_f16(w[0], w[1]);
          qv[i][2 * h + 1] = codes_f16(w[2], w[3]);
        }
        if (DEPTH) qs[i] = *(const f32x4_t*)(sqs + 16 * NS * wn + 16 * i + 4 * lg);
      }
#pragma unroll
      for (int j = 0; j < SUB; ++j) {
        f16x8_t pv[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const i32x4_t w = lds16(sb + p_rd[h] + j * 2048);
          pv[2 * h] = codes_f16(w[0], w[1]);
          pv[2 * h + 1] = codes_f16(w[2], w[3]);
        }
        const float s = sps[prow + 16 * j] * wsc;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          f32x4_t pr = zero;
#pragma unroll
          for (int h = 0; h < 4; ++h) pr = __builtin_amdgcn_mfma_f32_16x16x32_f16(qv[i][h], pv[h], pr, 0, 0, 0);
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[i][j][v] += pr[v] * (DEPTH ? qs[i][v] * s : s);
        }
      }
    }
  };
  // Returns the blocks of 16 rows that the wave stored with NS instructions
  // each, -1 where their number is another (a ragged edge, sums).
  const auto store = [&](const Item& t) {
    const int blocks = min(max((t.rows - 16 * SUB * wm + 15) / 16, 0), SUB);
    if (DEPTH && !a.add && t.cols == C::BN) {
      // lanes lr and lr ^ 8 exchange halves, so that a store writes whole lines
      // of 128 bytes of 8 rows (half lines of 16 took 4% longer for the gradients
      // above; with 16-bit results it changes nothing); once, and more than the
      // caches hold, so past them (3% longer without)
      const bool low = lr < 8;
      const int r = 16 * SUB * wm + (lr & 7);
      float* const to = (float*)a.out + (t.e * a.R + t.r0 + r) * a.ldo + t.c0 + 16 * NS * wn + (low ? 0 : 16) + 4 * lg;
#pragma unroll
      for (int j = 0; j < SUB; ++j) {
        if (j >= blocks) break;
#pragma unroll
        for (int i = 0; i < NS; i += 2) {
          f32x4u_t up, down;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float mine = low ? acc[i][j][u] : acc[i + 1][j][u];
            const float other = dpp<0x128>(low ? acc[i + 1][j][u] : acc[i][j][u]);
            up[u] = low ? mine : other;
            down[u] = low ? other : mine;
          }
          float* const at = to + 16 * j * a.ldo + 16 * i;
          if (r + 16 * j < t.rows) __builtin_nontemporal_store(up, (f32x4u_t*)at);
          if (r + 16 * j + 8 < t.rows) __builtin_nontemporal_store(down, (f32x4u_t*)(at + 8 * a.ldo));
        }
      }
      return min(max((t.rows - 16 * SUB * wm + 7) / 16, 0), SUB);      // a last one of 8 rows has half the stores
    }
    int r_first = prow;
    asm volatile("" : "+v"(r_first));            // addresses made here: held through the products they spill (191 us, 180)
#pragma unroll
    for (int j = 0; j < SUB; ++j) {
      if (j >= blocks) break;
      const int r = r_first + 16 * j;
      if (r >= t.rows) continue;
      const int64_t at = (DEPTH ? t.e * a.R + t.r0 + r : t.r0 + r) * a.ldo + t.c0;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const int c = 16 * NS * wn + 16 * i + 4 * lg, n = t.cols - c;
        f32x4_t v = acc[i][j];
        if (DEPTH && a.add)
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (u < n) v[u] += ((const float*)a.out)[at + c + u];
        if (n >= 4) {
          if (DEPTH) {
            __builtin_nontemporal_store(f32x4u_t{v[0], v[1], v[2], v[3]}, (f32x4u_t*)((float*)a.out + at + c));
          } else if (a.otype == MOE_T_F32) {
            __builtin_memcpy((float*)a.out + at + c, &v, 16);
          } else {
            const uint2 w = a.otype == MOE_T_BF16 ? uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])}
                                                  : uint2{pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3])};
            __builtin_memcpy((uint16_t*)a.out + at + c, &w, 8);
          }
        } else {
#pragma unroll
          for (int u = 0; u < 3; ++u)
            if (u < n) store_value(a.out, at + c + u, a.otype, v[u]);
        }
      }
    }
    return t.cols == C::BN && !DEPTH ? blocks : -1;
  };
  // Loads and stores are counted in the order of issue.  The unit that is
  // waited for was loaded before `newer` other units and, for NST - 1 units
  // after an item's end, before its stores: those stay outstanding.
  // Fewer may stay outstanding than could: near the end, and beside a ragged
  // item's stores.
  const auto wait = [&](int newer, int stored) {
    constexpr int UNITS = (C::LOADS + 1) * (C::NST - 2);
    static_assert(UNITS + NS * SUB < 64, "the counter's range");
    if (newer < C::NST - 2) wait_vmcnt<0>();
    else if (stored >= SUB) wait_vmcnt<UNITS + NS * SUB>();
    else if (stored >= SUB / 2) wait_vmcnt<UNITS + NS * SUB / 2>();
    else wait_vmcnt<UNITS>();
  };

  // ---- the stream -----------------------------------------------------------
  // (item, group) units in turn; loads run NST - 1 units ahead.
  Item cur, nxt;
  decode(it, cur);
  nxt = cur;
  int nit = it;
  int ng = cur.g0;
  bool more = true;                              // nxt, ng: the next unit to load
  const auto settle = [&] {                      // to an item that has groups
    while (more && ng >= nxt.g1) {
      nit += per;
      if (nit >= it1) {
        more = false;
        break;
      }
      decode(nit, nxt);
      ng = nxt.g0;
      aim(nxt);
    }
  };
  aim(nxt);
  settle();
  clear();
  int ahead = 0, in = 0, out = 0;                // units in flight, stage to fill, stage to read
  int stored = 0, since = 0;                     // blocks of the last item, units since
  const auto advance = [&] {
    if (!more) return;
    issue(ng, in);
    in = in + 1 == C::NST ? 0 : in + 1;
    ++ahead;
    ++ng;
    settle();
  };
#pragma unroll
  for (int i = 0; i < C::NST - 1; ++i) advance();
  for (;;) {
    for (int g = cur.g0; g < cur.g1; ++g) {
      wait(ahead - 1, since < C::NST - 1 ? stored : 0);
      ++since;
      barrier_keep_loads();                      // the unit is there, and the stage before it is free
      __builtin_amdgcn_sched_barrier(0);
      advance();
      --ahead;
      if (cur.rows > 16 * SUB * wm) compute(lds + out * C::STAGE);
      out = out + 1 == C::NST ? 0 : out + 1;
    }
    stored = max(store(cur), 0);
    since = 0;
    it += per;
    if (it >= it1) break;
    decode(it, cur);
    clear();
  }
}

constexpr int64_t MAX_SIZE = 1 << 30, MAX_MATRIX = (int64_t)1 << 40;
constexpr int CUS = 256;

// Sum of the parts of a split gradient, in their order.
__global__ void __launch_bounds__(256)
join_kernel(const float* __restrict__ part, int split, int64_t rows, int64_t R, int64_t C, float* __restrict__ out,
            int64_t ldo, int add) {
  const int64_t units = (C + 3) / 4, at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = at / units, c = (at - row * units) * 4;
  if (row >= rows) return;
  const int64_t e = row / R, r = row - e * R;
  float v[4] = {};
  const int n = (int)min((int64_t)4, C - c);
  for (int s = 0; s < split; ++s) {
    const float* p = part + ((e * split + s) * R + r) * C + c;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) v[i] += p[i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) out[row * ldo + c + i] = (add ? out[row * ldo + c + i] : 0.0f) + v[i];
}

template <int RT>
int launch_stream(const MmArgs& m, hipStream_t s) {
  const int64_t blocks = (m.R + 16 * RT - 1) / (16 * RT) + (m.offsets ? std::min<int64_t>(m.E, m.R) : 0);
  const dim3 grid((unsigned)((m.C + 15) / 16), (unsigned)std::min<int64_t>(blocks, 65535));
  stream_kernel<RT><<<grid, 64 * STREAM_WAVES, 0, s>>>(m, (int)blocks);
  return launched();
}

template <bool DEPTH, bool EXACT, int SUB, int NS>
int launch_tiles(const MmArgs& m, hipStream_t s) {
  using C = Tile<DEPTH, EXACT, SUB, NS>;
  const hipError_t e = hipFuncSetAttribute((const void*)tile_kernel<DEPTH, EXACT, SUB, NS>,
                                           hipFuncAttributeMaxDynamicSharedMemorySize, C::LDS);
  if (e != hipSuccess) return bad(MOE_E_HIP, hipGetErrorString(e));
  const int64_t mt = (m.R + C::BM - 1) / C::BM + (!DEPTH && m.offsets ? std::min<int64_t>(m.E, m.R) : 0);
  const int64_t items = mt * ((m.C + C::BN - 1) / C::BN) * (DEPTH ? (int64_t)m.E * m.split : 1);
  if (items > I32_MAX) return bad(MOE_E_UNSUPPORTED, "too many values");
  const unsigned grid = (unsigned)std::min<int64_t>((items + 7) / 8 * 8, CUS);
  tile_kernel<DEPTH, EXACT, SUB, NS><<<grid, 512, C::LDS, s>>>(m);
  return launched();
}

// What a call would take: rounds of the card's 256 workgroups, times the
// groups of the summed axis, times what one group takes (ns, measured at 4096
// columns of Q and groups enough to hide the ends):
//   tile                    64x128  128x128  128x256  256x256
//   8-bit instruction          760     1020     1470     2500 (experts 2900)
//   exact                      930     1330     2150
//   exact, row scales          890     1350     2050
//   few rows          16 rows: 190  32: 270  64: 390
// It is right within a tenth where the rows are (dense, 4096 inputs, us, both
// sides of each change): 4096 columns, 128 rows: 26 as few rows, 24 as 64x128;
// 512 rows 25 / 32 as 128x128; 1024 rows 48 as 64x128 / 34 / 46 as 128x256;
// 2048 rows 65 as 128x128 / 50 / 80 as 256x256; 1024 columns, 512 rows: 25 as
// few rows, 24 as 64x128.  Experts' rows are expected to fill their last tile
// by half, and only their capacity is known here, not the rows in use: one
// token of 8 of 128 experts, 2048 x 1536, takes 22 us on segments padded to 128
// (1024 rows to the rule) and 14 without padding, 4, 32 and 128 tokens the same
// on both; where the weights' bytes are the time, the table does not say it
// (4096 tokens of 256 experts: 1690 by it, 1000 taken).  Measured choices: 64
// experts of about 96 rows, 2048 x 2048: 112 / 97 / 90 / 96; 128 of about 512
// rows, unevenly, 1536 x 2048: 400 as 128x256 / 461 as 256x256, which leaves
// more of its last tiles empty.
double rounds(double workgroups) { return std::ceil(workgroups / CUS); }

double row_tiles(const MmArgs& m, bool depth, int BM) {
  if (depth || !m.offsets) return (double)((m.R + BM - 1) / BM);
  const double act = (double)std::min<int64_t>(m.E, m.R);
  return act * std::max(1.0, (double)m.R / act / BM + 0.5);
}

double tile_cost(const MmArgs& m, bool depth, int BM, int BN, double ns, double groups) {
  return rounds(row_tiles(m, depth, BM) * ((m.C + BN - 1) / BN) * (depth ? (double)m.E * m.split : 1.0)) * groups * ns;
}

int product(const MmArgs& m, hipStream_t s) {
  const bool exact = m.otype != MOE_T_BF16;
  const double G = m.groups;
  struct Choice {
    double cost;
    int (*launch)(const MmArgs&, hipStream_t);
  };
  // few rows of an expert: a workgroup looks its rows up first, about 3 us
  const auto stream = [&](int rows, double ns) {
    return rounds(row_tiles(m, false, rows) * ((m.C + 15) / 16)) * (G * ns + (m.offsets ? 3000.0 : 0.0));
  };
  const Choice choices[] = {
      {stream(16, 190), launch_stream<1>},
      {stream(32, 270), launch_stream<2>},
      {stream(64, 390), launch_stream<4>},
      {tile_cost(m, false, 64, 128, exact ? 930 : 760, G),
       exact ? launch_tiles<false, true, 2, 2> : launch_tiles<false, false, 2, 2>},
      {tile_cost(m, false, 128, 128, exact ? 1330 : 1020, G),
       exact ? launch_tiles<false, true, 4, 2> : launch_tiles<false, false, 4, 2>},
      {tile_cost(m, false, 128, 256, exact ? 2150 : 1470, G),
       exact ? launch_tiles<false, true, 4, 4> : launch_tiles<false, false, 4, 4>},
      {exact ? 1e300 : tile_cost(m, false, 256, 256, m.offsets ? 2900 : 2500, G), launch_tiles<false, false, 8, 4>},
  };
  const Choice* best = choices;
  for (const Choice& c : choices)
    if (c.cost < best->cost) best = &c;
  return best->launch(m, s);
}

// Tile and parts of a gradient.  Parts are written and read again, at about
// 4 bytes a ps.
struct Depth {
  int shape, split;
};
Depth choose_depth(int64_t E, int64_t N, int64_t K, int64_t rows) {
  static const struct {
    int BM, BN;
    double ns;
  } shapes[] = {{64, 128, 890}, {128, 128, 1350}, {128, 256, 2050}};
  MmArgs m{};
  m.E = (int)E;
  m.R = N;
  m.C = K;
  const double G = std::max(1.0, std::ceil((double)((rows + 127) / 128) / (double)E));      // of an expert
  Depth best{0, 1};
  double least = 1e300;
  for (int split = 1; split <= 16 && split <= G; split *= 2)
    for (int i = 0; i < 3; ++i) {
      m.split = split;
      const double join = split > 1 ? 3000.0 + (2.0 * split + 1) * E * N * K * 4 / 4000.0 : 0.0;
      const double cost = tile_cost(m, true, shapes[i].BM, shapes[i].BN, shapes[i].ns, std::ceil(G / split)) + join;
      if (cost < least) {
        least = cost;
        best = Depth{i, split};
      }
    }
  return best;
}

bool gradient_sizes(int64_t E, int64_t rows, int64_t N, int64_t K) {
  return E >= 1 && E <= MAX_E && rows >= 0 && rows <= MAX_SIZE && N >= 1 && N <= MAX_SIZE && K >= 1 && K <= MAX_SIZE &&
         N * K <= MAX_MATRIX;
}

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
  const MmArgs m{a, a_scales, w, w_scales, offsets, counts, (int)E, rows, N, K, (int)G, out, ldo, otype, 0, 1};
  return product(m, (hipStream_t)stream);
}

size_t moe_fp8_weight_gradient_workspace_bytes(int64_t E, int64_t rows, int64_t N, int64_t K) {
  if (!gradient_sizes(E, rows, N, K)) return 0;
  const int split = choose_depth(E, N, K, rows).split;
  return split > 1 ? (size_t)split * E * N * K * 4 : 0;
}

int moe_fp8_weight_gradient(const uint8_t* dy_t, const float* dy_scales, const uint8_t* x_t, const float* x_scales,
                            const int32_t* offsets, int64_t E, int64_t rows, int64_t N, int64_t K, int add, float* dw,
                            int64_t ldw, void* ws, size_t ws_bytes, void* stream) {
  if (rows < 0 || rows > I32_MAX) return bad(MOE_E_INVAL, "rows outside [0, 2^31)");
  if (E < 1 || E > MAX_E) return bad(MOE_E_INVAL, "need 1 <= E <= 1024");
  if (!offsets && E != 1) return bad(MOE_E_INVAL, "without offsets: one matrix");
  if (N < 1 || K < 1) return bad(MOE_E_INVAL, "need N >= 1 and K >= 1");
  if (!gradient_sizes(E, rows, N, K))
    return bad(MOE_E_UNSUPPORTED, "more than 2^30 rows or columns, or a matrix of more than 2^40 values");
  if (ldw < K) return bad(MOE_E_INVAL, "dw's row stride smaller than its width");
  if (ldw > ((int64_t)1 << 40)) return bad(MOE_E_UNSUPPORTED, "dw's row stride over 2^40");
  if (!dw || (rows && (!dy_t || !dy_scales || !x_t || !x_scales))) return bad(MOE_E_INVAL, "null argument");
  if (((uintptr_t)dy_t | (uintptr_t)x_t) % 16) return bad(MOE_E_INVAL, "codes start on 16 bytes");
  const Depth d = choose_depth(E, N, K, rows);
  const size_t need = d.split > 1 ? (size_t)d.split * E * N * K * 4 : 0;
  if (need && (!ws || ws_bytes < need))
    return bad(MOE_E_INVAL, "workspace smaller than moe_fp8_weight_gradient_workspace_bytes");
  if (need && (uintptr_t)ws % 4) return bad(MOE_E_INVAL, "the workspace holds floats: it starts on 4 bytes");
  const int64_t Rp = (rows + 127) / 128 * 128, G = Rp / 128;
  const int64_t join_blocks = (E * N * ((K + 3) / 4) + 255) / 256;
  if (need && join_blocks > MAX_BLOCKS) return bad(MOE_E_UNSUPPORTED, "too many values");
  if (outputs_shared({row_span(dw, E * N, K, ldw, 4), span(need ? ws : nullptr, (int64_t)need)},
                     {span(dy_t, N * Rp), span(dy_scales, G * N * 4), span(x_t, K * Rp), span(x_scales, G * K * 4),
                      span(offsets, (E + 1) * 4)}))
    return shared();
  const hipStream_t s = (hipStream_t)stream;
  const MmArgs m{dy_t, dy_scales, x_t, x_scales, offsets, nullptr, (int)E, N, K, Rp, (int)G, need ? ws : dw,
                 need ? K : ldw, MOE_T_F32, need ? 0 : add, d.split};
  const int rc = d.shape == 0 ? launch_tiles<true, true, 2, 2>(m, s)
                              : d.shape == 1 ? launch_tiles<true, true, 4, 2>(m, s) : launch_tiles<true, true, 4, 4>(m, s);
  if (rc || !need) return rc;
  join_kernel<<<(unsigned)join_blocks, 256, 0, s>>>((const float*)ws, d.split, E * N, N, K, dw, ldw, add);
  return launched();
}

}  // extern "C"
