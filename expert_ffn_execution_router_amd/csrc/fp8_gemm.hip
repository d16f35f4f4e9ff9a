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
template <bool DEPTH, bool EXACT, int SUB, int NS>
struct Tile {
  static constexpr int BM = 32 * SUB, BN = 64 * NS;
  static constexpr int LOADS = (BM + BN) / 64;             // 1 KiB blocks of 8 rows for each wave
  static constexpr int P_OFF = 0, Q_OFF = BM * 128;
  static constexpr int SP_OFF = Q_OFF + BN * 128;          // scales: 64 floats a wave, 8 waves
  static constexpr int STAGE = SP_OFF + 8 * 256;
  static constexpr int NST = 3 * STAGE + 4352 <= 160 * 1024 ? 3 : 2;
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
  const int64_t nitems = (int64_t)nm_all * ntiles * (DEPTH ? a.E : 1);
  // each XCD deals its eighth of the list to its workgroups in turn
  constexpr int N_XCD = 8;
  const int xcd = blockIdx.x % N_XCD, per = (gridDim.x + N_XCD - 1 - xcd) / N_XCD;
  const int64_t it1 = (xcd + 1) * nitems / N_XCD;
  int64_t it = xcd * nitems / N_XCD + blockIdx.x / N_XCD;
  if (it >= it1) return;

  // The list goes expert by expert, four column tiles at a time over the
  // row tiles, so that workgroups side by side share both.
  const auto decode = [&](int64_t i, Item& o) {
    int e = 0, nm = dense_m;
    int64_t q = i;
    int64_t first = 0, end = a.R;
    o.g0 = 0;
    o.g1 = a.groups;
    if (DEPTH) {
      e = (int)(i / ((int64_t)dense_m * ntiles));
      q = i - (int64_t)e * dense_m * ntiles;
      if (a.offsets) {
        o.g0 = min(max(a.offsets[e], 0) / 128, a.groups);
        o.g1 = max(min(max(a.offsets[e + 1], 0) / 128, a.groups), o.g0);
      }
    } else if (a.offsets) {
      const int m = (int)(i / ntiles);
      int hi = a.E - 1;
      while (e < hi) {
        const int mid = (e + hi + 1) >> 1;
        if (pref[mid] <= m) e = mid; else hi = mid - 1;
      }
      nm = pref[e + 1] - pref[e];
      q = i - (int64_t)pref[e] * ntiles;
      first = min(max((int64_t)a.offsets[e], (int64_t)0), a.R);
      const int64_t many = a.counts ? (int64_t)a.counts[e] : (int64_t)a.offsets[e + 1] - a.offsets[e];
      end = max(min(first + many, a.R), first);
    }
    const int quad = (int)(q / (4 * nm)), rest = (int)(q - (int64_t)quad * 4 * nm), wide = min(4, ntiles - 4 * quad);
    const int mt = rest / wide, nt = 4 * quad + rest - mt * wide;
    // equal tiles of the rows there are
    const int64_t step = ((end - first + nm - 1) / nm + 15) / 16 * 16;
    const int64_t r0 = first + mt * step;
    o.e = __builtin_amdgcn_readfirstlane(e);
    o.rows = __builtin_amdgcn_readfirstlane((int)max(min(step, end - r0), (int64_t)0));
    const int64_t c0 = (int64_t)nt * C::BN;
    o.cols = __builtin_amdgcn_readfirstlane((int)min((int64_t)C::BN, a.C - c0));
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
  const auto store = [&](const Item& t) {
#pragma unroll
    for (int j = 0; j < SUB; ++j) {
      const int r = prow + 16 * j;
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
          if (a.otype == MOE_T_F32) {
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
  };

  // ---- the stream -----------------------------------------------------------
  // (item, group) units in turn; loads run NST - 1 units ahead.
  Item cur, nxt;
  decode(it, cur);
  nxt = cur;
  int64_t nit = it;
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
      if (C::NST == 3 && ahead == 2) wait_vmcnt<C::LOADS + 1>();
      else wait_vmcnt<0>();
      barrier_keep_loads();                      // the unit is there, and the stage before it is free
      __builtin_amdgcn_sched_barrier(0);
      advance();
      --ahead;
      if (cur.rows > 16 * SUB * wm) compute(lds + out * C::STAGE);
      out = out + 1 == C::NST ? 0 : out + 1;
    }
    store(cur);
    it += per;
    if (it >= it1) break;
    decode(it, cur);
    clear();
  }
}

constexpr int64_t MAX_SIZE = 1 << 30, MAX_MATRIX = (int64_t)1 << 40;

template <bool DEPTH, bool EXACT, int SUB, int NS>
int launch_tiles(const MmArgs& m, hipStream_t s) {
  using C = Tile<DEPTH, EXACT, SUB, NS>;
  const hipError_t e = hipFuncSetAttribute((const void*)tile_kernel<DEPTH, EXACT, SUB, NS>,
                                           hipFuncAttributeMaxDynamicSharedMemorySize, C::LDS);
  if (e != hipSuccess) return bad(MOE_E_HIP, hipGetErrorString(e));
  const int64_t mt = (m.R + C::BM - 1) / C::BM + (!DEPTH && m.offsets ? std::min<int64_t>(m.E, m.R) : 0);
  const int64_t items = mt * ((m.C + C::BN - 1) / C::BN) * (DEPTH ? m.E : 1);
  const unsigned grid = (unsigned)std::min<int64_t>((items + 7) / 8 * 8, 256);
  tile_kernel<DEPTH, EXACT, SUB, NS><<<grid, 512, C::LDS, s>>>(m);
  return launched();
}

// Tiles of BM x BN of a call.
int64_t tiles_of(const MmArgs& m, bool depth, int BM, int BN) {
  return (m.R + BM - 1) / BM * ((m.C + BN - 1) / BN) * (depth ? m.E : 1);
}

template <bool DEPTH, bool EXACT>
int choose_tiles(const MmArgs& m, hipStream_t s) {
  constexpr int CUS = 256;
  const int64_t per_expert = DEPTH || !m.offsets ? m.R : m.R / m.E;
  if constexpr (!EXACT)
    if (per_expert > 192 && tiles_of(m, DEPTH, 256, 256) >= CUS) return launch_tiles<DEPTH, EXACT, 8, 4>(m, s);
  if (tiles_of(m, DEPTH, 128, 256) >= CUS) return launch_tiles<DEPTH, EXACT, 4, 4>(m, s);
  if (tiles_of(m, DEPTH, 128, 128) >= CUS) return launch_tiles<DEPTH, EXACT, 4, 2>(m, s);
  return launch_tiles<DEPTH, EXACT, 2, 2>(m, s);
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
  const MmArgs m{a, a_scales, w, w_scales, offsets, counts, (int)E, rows, N, K, (int)G, out, ldo, otype, 0};
  if (rows > 64) return otype == MOE_T_F32 ? choose_tiles<false, true>(m, (hipStream_t)stream) : choose_tiles<false, false>(m, (hipStream_t)stream);
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
  return choose_tiles<true, true>(m, (hipStream_t)stream);
}

}  // extern "C"
