// Values to E4M3 codes with a scale for each group of 128 (rows, the same
// transposed, blocks of weights), and the gradient of silu(gate) * up.
#include "e4m3.h"
#include "op_host.h"

namespace {

struct QuantArgs {
  const void* x;
  int64_t ldx, x_rows, x_step;     // x_step: values from one matrix to the next (weights)
  const int32_t* row_map;
  int map_div;
  uint32_t div_mul;                // n / map_div = n div_mul >> div_shift, for n < 2^31 (n without map_div)
  int div_shift;
  int64_t R, K;
  uint8_t* codes;                  // [R][Kp]
  float* scales;                   // rows: [Kp/128][R]; weights: [Rp/128][Kp/128]
  uint8_t* codes_t;                // [K][Rp]
  float* scales_t;                 // rows: [Rp/128][K]; weights: [Kp/128][Rp/128]
  int row_tiles, col_tiles;
};

enum { Q_ROWS = 1, Q_COLS = 2, Q_BLOCKS = 4 };

// A workgroup takes 128 x 128 values: thread (q, l) = (tid / 16, tid % 16)
// holds rows 4q .. 4q+3 of columns 8l .. 8l+7, so a row's group is a row of 16
// lanes and a column's four codes of a thread are a word of the transposed
// row.  Transposed codes pass through LDS, so that whole rows of 128 bytes are
// stored: the 16-byte pieces of column c are XORed with c / 8, which spreads
// the words that a wave writes over the banks.
// The bytes are the floor, the vector instructions (about 11 for a value of
// gathered rows, 18 before scales were shared and loads freed of branches) and
// the chain map, row, store the bound: 24576 gathered rows of 4096 bf16 in 32768
// 69 us (138 MB that must move; x is read six times, from the caches), 9001
// gated rows 16.0 us (2.6 TB/s), 65536 rows of 1536 in padded segments both ways
// 80 us (about 430 MB, 5.3 TB/s); 8192 x 4096 bf16, in the caches, 16.8 us as rows,
// 17.4 transposed, 22.2 both ways; weights of 32 x 4096 x 4096 bf16 279 us (5.8
// TB/s), both ways 378.
// 512 columns by 16 rows to a workgroup took 75 us for the gathered rows, and
// tiles in column order, which halve the bytes fetched, the same 72 as in row
// order then.
constexpr int Q_THREADS = 512, Q_SPAN = 4;       // rows of a thread

DEV int tile_word(int c, int q) { return c * 32 + (((q >> 2) ^ (c >> 3)) & 7) * 4 + (q & 3); }

__device__ const uint4 NOTHING[2] = {};          // eight zeros of any type

template <int DT, int MODE, bool GATED>
__global__ void __launch_bounds__(Q_THREADS)
quant_kernel(QuantArgs a) {
  typedef typename Elem<DT>::type T;
  constexpr int WAVES = Q_THREADS / 64, S = Q_SPAN;
  __shared__ float part[WAVES][128];
  __shared__ __align__(16) uint32_t tile[(MODE & Q_ROWS) && !(MODE & Q_COLS) ? 4 : 128 * 32];
  const int tid = threadIdx.x, q = tid >> 4, l = tid & 15, wave = tid >> 6;
  const unsigned ct = blockIdx.x % (unsigned)a.col_tiles, rest = blockIdx.x / (unsigned)a.col_tiles;
  const unsigned rt = rest % (unsigned)a.row_tiles, e = rest / (unsigned)a.row_tiles;
  const int r0 = (int)rt * 128 + S * q, c0 = (int)ct * 128 + 8 * l, R = (int)a.R;
  const int64_t Kp = (int64_t)a.col_tiles * 128, Rp = (int64_t)a.row_tiles * 128;
  const T* x = (const T*)a.x + e * a.x_step;
  float v[S][8], u[S][8];
  unsigned keep = 0;               // bit i: row i is written
  int src[S];                      // its row of x, -1: zeros
  int m[S];
#pragma unroll
  for (int i = 0; i < S; ++i) m[i] = r0 + i;
  if (a.row_map)
#pragma unroll
    for (int i = 0; i < S; ++i) m[i] = a.row_map[min(r0 + i, R - 1)];
#pragma unroll
  for (int i = 0; i < S; ++i) {
    const uint32_t n = a.map_div ? (uint32_t)m[i] : (uint32_t)(r0 + i);
    const int at = (int)((uint64_t)n * a.div_mul >> a.div_shift);
    if (r0 + i < R && m[i] >= -1) keep |= 1u << i;
    src[i] = r0 + i < R && m[i] >= 0 && at < (int)a.x_rows ? at : -1;
  }
  if ((int64_t)ct * 128 + 128 <= a.K) {
    Pack<T, 8> raw[S], raw_u[S];   // loads without a branch between them
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const T* from = x + (uint64_t)(uint32_t)src[i] * (uint64_t)a.ldx + c0;
      const T* up = from + a.K;
      from = src[i] >= 0 ? from : (const T*)NOTHING;
      up = src[i] >= 0 ? up : (const T*)NOTHING;
      __builtin_memcpy(&raw[i], from, sizeof(raw[i]));
      if (GATED) __builtin_memcpy(&raw_u[i], up, sizeof(raw_u[i]));
    }
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[i][j] = Elem<DT>::load(raw[i].v[j]);
        if (GATED) u[i][j] = Elem<DT>::load(raw_u[i].v[j]);
      }
  } else {
#pragma unroll
    for (int i = 0; i < S; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = u[i][j] = 0.0f;
      if (src[i] < 0) continue;
      load8<DT>(x + (int64_t)src[i] * a.ldx, c0, a.K, v[i]);
      if (GATED) load8<DT>(x + (int64_t)src[i] * a.ldx + a.K, c0, a.K, u[i]);
    }
  }
  if (GATED)
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = silu(v[i][j]) * u[i][j];
  // the words of the transposed codes to their rows
  const auto store_t = [&](uint8_t* to) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 128 * 8 / Q_THREADS; ++i) {
      const int at = i * Q_THREADS + tid, c = at >> 3, p = at & 7;
      const int64_t col = (int64_t)ct * 128 + c;
      if (col < a.K)
        *(i32x4_t*)(to + col * Rp + (int64_t)rt * 128 + 16 * p) = *(const i32x4_t*)(tile + tile_word(c, 4 * p));
    }
  };
  if (MODE & Q_ROWS) {
    // lane 4 n + i of a group takes over row i of its quad, joins it with the
    // other quads' and gives the scales back: two divisions in place of eight
    static_assert(S == 4, "a row for each lane of a quad");
    float mx[S];
#pragma unroll
    for (int i = 0; i < S; ++i) mx[i] = abs_max(v[i]);
    const bool odd = l & 1, high = l & 2;
    const float lo = maximum(odd ? mx[1] : mx[0], dpp<0xB1>(odd ? mx[0] : mx[1]));
    const float hi = maximum(odd ? mx[3] : mx[2], dpp<0xB1>(odd ? mx[2] : mx[3]));
    float m4 = maximum(high ? hi : lo, dpp<0x4E>(high ? lo : hi));
    m4 = maximum(m4, dpp<0x124>(m4));
    m4 = maximum(m4, dpp<0x128>(m4));
    const GroupScale s = group_scale(m4);
    const float inv[S] = {quad_lane<0>(s.inv), quad_lane<1>(s.inv), quad_lane<2>(s.inv), quad_lane<3>(s.inv)};
    uint8_t* to = a.codes + (int64_t)r0 * Kp + c0;
#pragma unroll
    for (int i = 0; i < S; ++i) {
      if (!((keep >> i) & 1)) continue;
      const uint2 w = {codes4(v[i][0], v[i][1], v[i][2], v[i][3], inv[i]),
                       codes4(v[i][4], v[i][5], v[i][6], v[i][7], inv[i])};
      *(uint2*)(to + i * Kp) = w;
    }
    if (l < S && ((keep >> l) & 1)) a.scales[(int64_t)ct * a.R + r0 + l] = s.scale;
  }
  if (MODE & Q_COLS) {
    if (a.row_map && !__syncthreads_or(keep != 0)) return;      // nothing but rows behind the last segment
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float mx = lanes_max(abs_max({v[0][j], v[1][j], v[2][j], v[3][j]}));
      if ((tid & 63) < 16) part[wave][8 * l + j] = mx;
    }
    __syncthreads();
    if (tid < 128) {
      float mx = part[0][tid];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) mx = maximum(mx, part[w][tid]);
      const GroupScale s = group_scale(mx);
      const int64_t col = (int64_t)ct * 128 + tid;
      if (col < a.K) a.scales_t[(int64_t)rt * a.K + col] = s.scale;
      part[0][tid] = s.inv;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = 8 * l + j;
      tile[tile_word(c, q)] = codes4(v[0][j], v[1][j], v[2][j], v[3][j], part[0][c]);
    }
    store_t(a.codes_t);
  }
  if (MODE & Q_BLOCKS) {
    float mx = abs_max(v[0]);
#pragma unroll
    for (int i = 1; i < S; ++i) mx = maximum(mx, abs_max(v[i]));
    mx = lanes_max(row16_max(mx));
    if ((tid & 63) == 0) part[wave][0] = mx;
    __syncthreads();
    mx = part[0][0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) mx = maximum(mx, part[w][0]);
    const GroupScale s = group_scale(mx);
    const int64_t blocks = (int64_t)a.row_tiles * a.col_tiles;
    if (a.codes) {
#pragma unroll
      for (int i = 0; i < S; ++i) {
        if (r0 + i >= a.R) continue;
        const uint2 w = {codes4(v[i][0], v[i][1], v[i][2], v[i][3], s.inv),
                         codes4(v[i][4], v[i][5], v[i][6], v[i][7], s.inv)};
        *(uint2*)(a.codes + ((int64_t)e * a.R + r0 + i) * Kp + c0) = w;
      }
      if (tid == 0) a.scales[e * blocks + (int64_t)rt * a.col_tiles + ct] = s.scale;
    }
    if (a.codes_t) {
#pragma unroll
      for (int j = 0; j < 8; ++j) tile[tile_word(8 * l + j, q)] = codes4(v[0][j], v[1][j], v[2][j], v[3][j], s.inv);
      if (tid == 0) a.scales_t[e * blocks + (int64_t)ct * a.row_tiles + rt] = s.scale;
      store_t(a.codes_t + (int64_t)e * a.K * Rp);
    }
  }
}

// dz = [da u s (1 + g (1 - s)), da g s] with s = 1 / (1 + e^-g) of z = [g, u].
// Eight columns of each to a thread, for whole 16-byte loads of 16-bit values;
// the bytes are the bound: 65536 rows of 2 x 768 bf16 in 96 us (5.2 TB/s).
template <int DT>
__global__ void __launch_bounds__(256)
gated_backward_kernel(const typename Elem<DT>::type* __restrict__ z, int64_t ldz,
                      const typename Elem<DT>::type* __restrict__ da, int64_t lda, int64_t R, int64_t I,
                      typename Elem<DT>::type* __restrict__ dz, int64_t lddz) {
  const int64_t units = (I + 7) / 8, at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t r = at / units, c = (at - r * units) * 8;
  if (r >= R) return;
  float g[8], u[8], d[8], dg[8], du[8];
  load8<DT>(z + r * ldz, c, I, g);
  load8<DT>(z + r * ldz + I, c, I, u);
  load8<DT>(da + r * lda, c, I, d);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float s = 1.0f / (1.0f + expf(-g[i]));
    dg[i] = d[i] * u[i] * (s * (1.0f + g[i] * (1.0f - s)));
    du[i] = d[i] * (g[i] * s);
  }
  store8<DT>(dz + r * lddz, c, I, dg);
  store8<DT>(dz + r * lddz + I, c, I, du);
}

template <int MODE, bool GATED>
int launch_quant(int dt, const QuantArgs& a, int64_t matrices, hipStream_t s) {
  const int64_t blocks = (int64_t)a.row_tiles * a.col_tiles * matrices;
  if (dt == MOE_T_BF16) quant_kernel<MOE_T_BF16, MODE, GATED><<<(unsigned)blocks, Q_THREADS, 0, s>>>(a);
  else if (dt == MOE_T_F16) quant_kernel<MOE_T_F16, MODE, GATED><<<(unsigned)blocks, Q_THREADS, 0, s>>>(a);
  else quant_kernel<MOE_T_F32, MODE, GATED><<<(unsigned)blocks, Q_THREADS, 0, s>>>(a);
  return launched();
}

int64_t pad128(int64_t n) { return (n + 127) / 128 * 128; }

constexpr int64_t MAX_SIZE = 1 << 30;
constexpr int64_t MAX_TILES = MAX_BLOCKS / 2;      // of 512 threads

}  // namespace

extern "C" {

int moe_fp8_quantize(int dtype, const void* x, int64_t ldx, int64_t x_rows, const int32_t* row_map, int64_t map_div,
                     int gated, int64_t rows, int64_t cols, uint8_t* codes, float* scales, uint8_t* codes_t,
                     float* scales_t, void* stream) {
  const int b = elem_bytes(dtype);
  if (!b) return bad(MOE_E_INVAL, "unknown type");
  if (rows < 0 || rows > I32_MAX || x_rows < 0) return bad(MOE_E_INVAL, "rows outside [0, 2^31)");
  if (x_rows > I32_MAX) return bad(MOE_E_UNSUPPORTED, "x has more than 2^31 - 1 rows");
  if (cols < 1) return bad(MOE_E_INVAL, "need cols >= 1");
  if (cols > MAX_SIZE || rows > MAX_SIZE) return bad(MOE_E_UNSUPPORTED, "more than 2^30 rows or columns");
  const int64_t width = gated ? 2 * cols : cols;
  if (ldx < width) return bad(MOE_E_INVAL, "row stride smaller than the width");
  if (row_map && (map_div < 0 || map_div > I32_MAX)) return bad(MOE_E_INVAL, "need 0 <= map_div < 2^31");
  if (!(row_map && map_div) && x_rows < rows) return bad(MOE_E_INVAL, "x has fewer rows than the codes");
  if (!codes && !codes_t) return bad(MOE_E_INVAL, "neither codes nor codes_t");
  if (!codes != !scales || !codes_t != !scales_t) return bad(MOE_E_INVAL, "codes and scales come together");
  if (rows == 0) return MOE_OK;
  if (x_rows && !x) return bad(MOE_E_INVAL, "null argument");
  if (((uintptr_t)codes | (uintptr_t)codes_t) % 16) return bad(MOE_E_INVAL, "codes start on 16 bytes");
  const int64_t Kp = pad128(cols), Rp = pad128(rows);
  const int64_t div = row_map && map_div ? map_div : 1;
  int log2 = 0;                    // ceil(log2(div)); with m = floor(2^(31 + log2) / div) + 1, m div - 2^(31 + log2) <= 2^log2
  while (((int64_t)1 << log2) < div) ++log2;
  const uint32_t div_mul = (uint32_t)((((uint64_t)1 << (31 + log2)) / (uint64_t)div) + 1);
  QuantArgs a{x, ldx, x_rows, 0, row_map, row_map ? (int)map_div : 0, div_mul, 31 + log2, rows, cols, codes, scales, codes_t, scales_t,
              (int)(Rp / 128), (int)(Kp / 128)};
  if ((int64_t)a.row_tiles * a.col_tiles > MAX_TILES) return bad(MOE_E_UNSUPPORTED, "too many values");
  if (outputs_shared({span(codes, rows * Kp), span(scales, Kp / 128 * rows * 4), span(codes_t, cols * Rp),
                      span(scales_t, Rp / 128 * cols * 4)},
                     {row_span(x, x_rows, width, ldx, b), span(row_map, rows * 4)}))
    return shared();
  const hipStream_t s = (hipStream_t)stream;
  if (!codes_t) return gated ? launch_quant<Q_ROWS, true>(dtype, a, 1, s) : launch_quant<Q_ROWS, false>(dtype, a, 1, s);
  if (!codes) return gated ? launch_quant<Q_COLS, true>(dtype, a, 1, s) : launch_quant<Q_COLS, false>(dtype, a, 1, s);
  return gated ? launch_quant<Q_ROWS | Q_COLS, true>(dtype, a, 1, s)
               : launch_quant<Q_ROWS | Q_COLS, false>(dtype, a, 1, s);
}

int moe_fp8_quantize_weights(int dtype, const void* w, int64_t E, int64_t N, int64_t K, uint8_t* codes, float* scales,
                             uint8_t* codes_t, float* scales_t, void* stream) {
  const int b = elem_bytes(dtype);
  if (!b) return bad(MOE_E_INVAL, "unknown type");
  if (E < 1 || E > I32_MAX || N < 1 || K < 1) return bad(MOE_E_INVAL, "need E, N, K >= 1");
  if (N > MAX_SIZE || K > MAX_SIZE) return bad(MOE_E_UNSUPPORTED, "more than 2^30 rows or columns");
  if (!codes && !codes_t) return bad(MOE_E_INVAL, "neither codes nor codes_t");
  if (!codes != !scales || !codes_t != !scales_t) return bad(MOE_E_INVAL, "codes and scales come together");
  if (!w) return bad(MOE_E_INVAL, "null argument");
  if (((uintptr_t)codes | (uintptr_t)codes_t) % 16) return bad(MOE_E_INVAL, "codes start on 16 bytes");
  const int64_t Kp = pad128(K), Np = pad128(N), blocks = Np / 128 * (Kp / 128);
  if (blocks > MAX_TILES || blocks * E > MAX_TILES) return bad(MOE_E_UNSUPPORTED, "too many values");
  if (outputs_shared({span(codes, E * N * Kp), span(scales, E * blocks * 4), span(codes_t, E * K * Np),
                      span(scales_t, E * blocks * 4)},
                     {span(w, E * N * K * b)}))
    return shared();
  const QuantArgs a{w, K, N, N * K, nullptr, 0, 0x80000001u, 31, N, K, codes, scales, codes_t, scales_t, (int)(Np / 128),
                    (int)(Kp / 128)};
  return launch_quant<Q_BLOCKS, false>(dtype, a, E, (hipStream_t)stream);
}

int moe_gated_backward(int dtype, const void* z, int64_t ldz, const void* da, int64_t lda, int64_t rows, int64_t I,
                       void* dz, int64_t lddz, void* stream) {
  const int b = elem_bytes(dtype);
  if (!b) return bad(MOE_E_INVAL, "unknown type");
  if (rows < 0 || rows > I32_MAX) return bad(MOE_E_INVAL, "rows outside [0, 2^31)");
  if (I < 1) return bad(MOE_E_INVAL, "need a width of at least 1");
  if (I > MAX_SIZE) return bad(MOE_E_UNSUPPORTED, "rows wider than 2^30");
  if (ldz < 2 * I || lda < I || lddz < 2 * I) return bad(MOE_E_INVAL, "row stride smaller than the width");
  if (rows == 0) return MOE_OK;
  if (!z || !da || !dz) return bad(MOE_E_INVAL, "null argument");
  const int64_t blocks = (rows * ((I + 7) / 8) + 255) / 256;
  if (blocks > MAX_BLOCKS) return bad(MOE_E_UNSUPPORTED, "too many values");
  if (outputs_shared({row_span(dz, rows, 2 * I, lddz, b)},
                     {row_span(z, rows, 2 * I, ldz, b), row_span(da, rows, I, lda, b)}))
    return shared();
#define GO(D)                                                                                                       \
  gated_backward_kernel<D><<<(unsigned)blocks, 256, 0, (hipStream_t)stream>>>(                                      \
      (const Elem<D>::type*)z, ldz, (const Elem<D>::type*)da, lda, rows, I, (Elem<D>::type*)dz, lddz)
  if (dtype == MOE_T_BF16) GO(MOE_T_BF16);
  else if (dtype == MOE_T_F16) GO(MOE_T_F16);
  else GO(MOE_T_F32);
#undef GO
  return launched();
}

}  // extern "C"
