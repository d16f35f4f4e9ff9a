// The norms around a block, with its gate and residual scale:
//
//   h    = alpha r + gate * (y / rms(y)) w,   rms(v) = sqrt(mean v^2 + eps)
//   next = (h / rms(h)) w'
//
// h is rounded to the residual's type once and next is the norm of what is
// stored, so one call gives what two would.  Without y, h is r alone (the norm
// before a block).  Backward, with dh and dn the gradients of h and next, n =
// h / rms(h), x = y / rms(y):
//
//   d  = dh + (dn w' - n mean(dn w' n)) / rms(h)        dw' = sum_t dn n
//   dr = alpha d          dgate = d x w (summed over what it was spread over)
//   dv = gate d           dw = sum_t dv x
//   dy = (dv w - x mean(dv w x)) / rms(y)
//
// A row is read once and held in registers, as units of 8 columns, by a wave or
// a workgroup (wider rows of the backward pass: twice).  All sums are fp32 in a
// fixed order.  The bytes are the bound: 8192 rows of 4096, bf16 with an fp32
// residual, take 82 us (403 MB, 4.9 TB/s, as a copy), their gradients 3.1 to
// 3.7 TB/s; one row of 2048 takes 3 us, a launch and two trips to memory.  The
// norm before a block, 8192 x 4096 bf16 in the caches: 22.9 us, 23.5 as codes;
// its gradients with dw 66 (3.0 TB/s), as 65536 x 512 91, 16384 x 2048 71, 4096 x
// 8192 89.
#include "e4m3.h"
#include "op_host.h"

namespace {

constexpr int MAX_COLS = 16384, MAX_BWD_COLS = 8192;

struct NormArgs {
  const void* y;
  int64_t ldy;
  const void* r;
  int64_t ldr;
  float alpha;
  const void* w;
  const void* gate;
  int64_t gr, gc;                 // gate strides (0: spread over the axis)
  void* h;
  int64_t ldh;
  const void* w2;
  void* next;
  int64_t ldn;
  float* scales;                  // next as codes
  int64_t T;
  int cols;
  float eps, eps2;
  bool w_f32, gate_f32;
};

struct NormBwdArgs {
  const void* dh;
  int64_t lddh;
  const void* y;
  int64_t ldy;
  float alpha;
  const void* w;
  const void* gate;
  int64_t gr, gc;
  const void* dn;
  int64_t lddn;
  const void* h;
  int64_t ldh;
  const void* w2;
  void* dy;
  int64_t lddy;
  void* dr;
  int64_t lddr;
  void* dgate;                    // spread over columns or whole
  int64_t dgr, dgc;
  float* part;                    // [sets][parts][cols]
  int set_w, set_w2, set_g;       // place of each column sum, -1: none
  int64_t T;
  int cols, parts;
  float eps, eps2;
  bool w_f32, gate_f32, dgate_f32;
};

// Sum over the wave, in all of its lanes: inside rows of 16 lanes, then over
// the rows; lane 63 has it.  (Exchanges through LDS, 36 for six sums, were a
// third of the backward pass.)
DEV float wave_total(float v) {
#define STEP(CTRL, ROWS) \
  v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, ROWS, 0xf, false));
  STEP(0x111, 0xf) STEP(0x112, 0xf) STEP(0x114, 0xf) STEP(0x118, 0xf) STEP(0x142, 0xa) STEP(0x143, 0xc)
#undef STEP
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

// Sum over the threads of a row: one wave, or all waves of the workgroup.
template <int TPR>
DEV float row_sum(float v, float* lds) {
  v = wave_total(v);
  if (TPR == 64) return v;
  __syncthreads();                               // lds is free again
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < TPR / 64; ++i) s += lds[i];
  return s;
}

// N such sums at once.
template <int TPR, int N>
DEV void row_sums(float (&v)[N], float (*lds)[16]) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = wave_total(v[k]);
  if (TPR == 64) return;
  __syncthreads();
  if ((threadIdx.x & 63) == 0)
#pragma unroll
    for (int k = 0; k < N; ++k) lds[k][threadIdx.x >> 6] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    v[k] = 0.0f;
#pragma unroll
    for (int i = 0; i < TPR / 64; ++i) v[k] += lds[k][i];
  }
}

// Columns c .. c+7 of a row, zeros from cols on.  EVEN (cols a multiple of 8):
// without a branch, so that a row's loads are in flight together.
template <int DT, bool EVEN>
DEV void load_row(const typename Elem<DT>::type* row, long c, long cols, float (&f)[8]) {
  if (!EVEN) return load8<DT>(row, c, cols, f);
  load_vals<DT, 8>(row + min(c, cols - 8), f);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = c < cols ? f[i] : 0.0f;
}

// The same as they are stored, without what waits for them: past cols (EVEN)
// they are other values of the row, which values() makes zeros.
template <int DT>
using Raw = Pack<typename Elem<DT>::type, 8>;

template <int DT, bool EVEN>
DEV Raw<DT> load_raw(const typename Elem<DT>::type* row, long c, long cols) {
  Raw<DT> r = {};
  if (EVEN) {
    __builtin_memcpy(&r, row + min(c, cols - 8), sizeof(r));
  } else if (c + 8 <= cols) {
    __builtin_memcpy(&r, row + c, sizeof(r));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < cols) r.v[i] = row[c + i];
  }
  return r;
}

template <int DT>
DEV void values(const Raw<DT>& r, bool inside, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = inside ? Elem<DT>::load(r.v[i]) : 0.0f;
}

template <int DT, bool EVEN>
DEV void load_param(const void* p, bool f32, long c, long cols, float (&f)[8]) {
  if (DT == MOE_T_F32 || f32) load_row<MOE_T_F32, EVEN>((const float*)p, c, cols, f);
  else load_row<DT, EVEN>((const typename Elem<DT>::type*)p, c, cols, f);
}

// The gate of row t, columns c .. c+7 (zeros past cols).
template <int DT, bool EVEN>
DEV void load_gate(const void* p, bool f32, int64_t t, int64_t gr, int64_t gc, long c, long cols, float (&f)[8]) {
  typedef typename Elem<DT>::type T;
  if (gc == 0) {
    const float g = DT == MOE_T_F32 || f32 ? ((const float*)p)[t * gr] : Elem<DT>::load(((const T*)p)[t * gr]);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = g;
  } else if (DT == MOE_T_F32 || f32) {
    load_row<MOE_T_F32, EVEN>((const float*)p + t * gr, c, cols, f);
  } else {
    load_row<DT, EVEN>((const T*)p + t * gr, c, cols, f);
  }
}

template <int DT, int RT, int TPR, int NV, bool EVEN>
__global__ void __launch_bounds__(TPR == 64 ? 256 : TPR)
norm_kernel(NormArgs a) {
  typedef typename Elem<DT>::type TD;
  typedef typename Elem<RT>::type TR;
  __shared__ float lds[16];
  const int u0 = TPR == 64 ? threadIdx.x & 63 : threadIdx.x;
  const int64_t t = TPR == 64 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  if (t >= a.T) return;
  const int cols = a.cols;
  const float inv_n = 1.0f / (float)cols;
  float h[NV][8];
  if (a.r) {
#pragma unroll
    for (int i = 0; i < NV; ++i) load_row<RT, EVEN>((const TR*)a.r + t * a.ldr, (u0 + i * TPR) * 8, cols, h[i]);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] *= a.alpha;
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = 0.0f;
  }
  if (a.y) {
    float y[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) load_row<DT, EVEN>((const TD*)a.y + t * a.ldy, (u0 + i * TPR) * 8, cols, y[i]);
    float rs = 1.0f;
    if (a.w) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) s += y[i][j] * y[i][j];
      rs = 1.0f / sqrtf(row_sum<TPR>(s, lds) * inv_n + a.eps);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const long c = (u0 + i * TPR) * 8;
      if (a.w) {
        float w[8];
        load_param<DT, EVEN>(a.w, a.w_f32, c, cols, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[i][j] = y[i][j] * rs * w[j];
      }
      if (a.gate) {
        float g[8];
        load_gate<DT, EVEN>(a.gate, a.gate_f32, t, a.gr, a.gc, c, cols, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[i][j] *= g[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] += y[i][j];
    }
  }
  if (a.h) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const long c = (u0 + i * TPR) * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = Elem<RT>::load(Elem<RT>::store(h[i][j]));
      if (c < cols) store8<RT>((TR*)a.h + t * a.ldh, c, cols, h[i]);
    }
  }
  if (!a.next) return;
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) s += (u0 + i * TPR) * 8 + j < cols ? h[i][j] * h[i][j] : 0.0f;
  const float rs = 1.0f / sqrtf(row_sum<TPR>(s, lds) * inv_n + a.eps2);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const long c = (u0 + i * TPR) * 8;
    float w[8];
    load_param<DT, EVEN>(a.w2, a.w_f32, c, cols, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) h[i][j] = c + j < cols ? h[i][j] * rs * w[j] : 0.0f;
    if (!a.scales) {
      if (c < cols) store8<DT>((TD*)a.next + t * a.ldn, c, cols, h[i]);
      continue;
    }
    const GroupScale q = group_scale(row16_max(abs_max(h[i])));
    if (c / 128 * 128 >= cols) continue;             // whole groups: the last one's tail is zeros
    const uint2 v = {codes4(h[i][0], h[i][1], h[i][2], h[i][3], q.inv),
                     codes4(h[i][4], h[i][5], h[i][6], h[i][7], q.inv)};
    *(uint2*)((uint8_t*)a.next + t * a.ldn + c) = v;
    if ((u0 & 15) == 0) a.scales[c / 128 * a.T + t] = q.scale;
  }
}

__device__ const uint4 NOTHING[2] = {};

template <typename T>
struct Rows {
  const T* p;
  int64_t ld;
  long cols;
  DEV Rows(const void* p, int64_t ld, long cols)
      : p(p ? (const T*)p : (const T*)NOTHING), ld(p ? ld : 0), cols(p ? cols : 8) {}
};

// With D = dn w', G = gate w and m = mean(D n): <d, G y> = <dh, G y> + (<D, G y>
// - m <h, G y> / rms(h)) / rms(h), so that one joint sum over the row, of values
// as they were read, gives both roots and both means.  HELD units of a thread
// stay in registers between that sum and the results; 0 (the widest rows):
// they are read again, and the column sums are kept in LDS, as neither fits
// without spilling registers.
template <int DT, int RT, int TPR, int HELD, bool EVEN>
__global__ void __launch_bounds__(TPR == 64 ? 256 : TPR)
norm_bwd_kernel(NormBwdArgs a) {
  typedef typename Elem<DT>::type TD;
  typedef typename Elem<RT>::type TR;
  constexpr bool WIDE = HELD == 0, AHEAD = HELD == 1;
  constexpr int NV = WIDE ? 1 : HELD;
  __shared__ float lds[6][16];
  extern __shared__ __align__(16) float lds_sums[];     // WIDE: [3][MAX_BWD_COLS]
  const int u0 = TPR == 64 ? threadIdx.x & 63 : threadIdx.x;
  const int part = TPR == 64 ? blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  const int cols = a.cols, units = WIDE ? (cols + 8 * TPR - 1) / (8 * TPR) : NV;
  const float inv_n = 1.0f / (float)cols;
  const auto column = [&](int i) { return (long)(u0 + i * TPR) * 8; };
  const auto each = [&](auto f) __attribute__((always_inline)) {
    if constexpr (WIDE) {
#pragma unroll 1
      for (int i = 0; i < units; ++i) f(i);
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) f(i);
    }
  };
  // column sums of the thread's units: dw, dw', dgate
  float sums[3][NV][8] = {};
  const auto count = [&](int k, int i, const float (&v)[8]) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (WIDE) lds_sums[k * MAX_BWD_COLS + column(i) + j] += v[j];
      else sums[k][i][j] += v[j];
    }
  };
  if (WIDE)
    each([&](int i) {
#pragma unroll
      for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) lds_sums[k * MAX_BWD_COLS + column(i) + j] = 0.0f;
    });
  struct Unit {
    Raw<RT> d, n;                                       // dh, h
    Raw<DT> g, x;                                       // dn, y
  };
  // What is not there is 8 zeros of every row: loads under a condition would be
  // waited for where its two sides meet.
  const Rows<TR> dh(a.dh, a.lddh, cols), h(a.dn ? a.h : nullptr, a.ldh, cols);
  const Rows<TD> dn(a.dn, a.lddn, cols), y(a.y, a.ldy, cols);
  const auto read = [&](int64_t t, int i, Unit& u) __attribute__((always_inline)) {
    u.d = load_raw<RT, EVEN>(dh.p + t * dh.ld, column(i), dh.cols);
    u.n = load_raw<RT, EVEN>(h.p + t * h.ld, column(i), h.cols);
    u.g = load_raw<DT, EVEN>(dn.p + t * dn.ld, column(i), dn.cols);
    u.x = load_raw<DT, EVEN>(y.p + t * y.ld, column(i), y.cols);
  };
  // AHEAD: the next row is on its way while one is worked on (a CU holds one
  // workgroup of 512), and what is the same for every row stays in registers,
  // as its loads would wait for that row.  4099 rows of 4096 bf16 with a gate
  // per column: 64 us with the join (202 MB, 3.1 TB/s); 118 without reading ahead
  // and with a sum after the other, 70 with the loads under conditions.
  float hw[NV][8], hf[NV][8], hk[NV][8];                // w, w', gate
  const auto weights = [&](int i, float (&w)[8], float (&f)[8]) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = f[j] = 1.0f;
    if (a.dn) load_param<DT, EVEN>(a.w2, a.w_f32, column(i), cols, f);
    if (a.w) load_param<DT, EVEN>(a.w, a.w_f32, column(i), cols, w);
  };
  const auto gate = [&](int64_t t, int i, float (&k)[8]) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) k[j] = 1.0f;
    if (a.gate) load_gate<DT, EVEN>(a.gate, a.gate_f32, t, a.gr, a.gc, column(i), cols, k);
  };
  Unit next[NV] = {}, cur[NV] = {};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (!AHEAD) continue;
    weights(i, hw[i], hf[i]);
    gate(0, i, hk[i]);
    if (part < a.T) read(part, i, next[i]);
  }
  for (int64_t t = part; t < a.T; t += a.parts) {
    if (AHEAD) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (a.gr) gate(t, i, hk[i]);
        cur[i] = next[i];
        if (t + a.parts < a.T) read(t + a.parts, i, next[i]);
      }
    } else if (!WIDE) {
#pragma unroll
      for (int i = 0; i < NV; ++i) read(t, i, cur[i]);
    }
    struct Values {
      float d[8], n[8], g[8], x[8], w[8], f[8], k[8];
    };
    const auto get = [&](int i, Values& v) __attribute__((always_inline)) {
      if (WIDE) read(t, i, cur[0]);
      const Unit& u = cur[WIDE ? 0 : i];
      values<RT>(u.d, column(i) < cols, v.d);
      values<RT>(u.n, column(i) < cols, v.n);
      values<DT>(u.g, column(i) < cols, v.g);
      values<DT>(u.x, column(i) < cols, v.x);
      if (!AHEAD) weights(i, v.w, v.f);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (AHEAD) {
          v.w[j] = hw[WIDE ? 0 : i][j];
          v.f[j] = hf[WIDE ? 0 : i][j];
          v.k[j] = hk[WIDE ? 0 : i][j];
        }
      }
      if (!AHEAD) gate(t, i, v.k);
    };
    // h^2, D h, y^2, dh G y, D G y, h G y
    float s[6] = {};
    each([&](int i) __attribute__((always_inline)) {
      Values v;
      get(i, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float D = v.g[j] * v.f[j], gy = v.x[j] * (v.w[j] * v.k[j]);
        s[0] += v.n[j] * v.n[j];
        s[1] += D * v.n[j];
        s[2] += v.x[j] * v.x[j];
        s[3] += v.d[j] * gy;
        s[4] += D * gy;
        s[5] += v.n[j] * gy;
      }
    });
    row_sums<TPR>(s, lds);
    const float rh = a.dn ? 1.0f / sqrtf(s[0] * inv_n + a.eps2) : 0.0f, m = rh * s[1] * inv_n;
    const float ry = a.w ? 1.0f / sqrtf(s[2] * inv_n + a.eps) : 1.0f;
    const float mean = a.w ? ry * (s[3] + rh * (s[4] - m * rh * s[5])) * inv_n : 0.0f;      // <d, G x>
    const bool row_sum_of_gate = a.dgate && !a.dgc;     // a gate per row: <d, w x>
    float dg[1] = {0.0f};
    each([&](int i) __attribute__((always_inline)) {
      const long c = column(i);
      Values v;
      get(i, v);
      float out[8];
      if (a.dn) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float n = v.n[j] * rh;
          out[j] = v.g[j] * n;
          v.d[j] += rh * (v.g[j] * v.f[j] - n * m);
        }
        if (a.set_w2 >= 0) count(1, i, out);
      }
      if (a.y) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v.x[j] *= ry;
          out[j] = v.d[j] * v.x[j] * v.k[j];
        }
        if (a.set_w >= 0) count(0, i, out);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          out[j] = v.d[j] * v.x[j] * v.w[j];
          dg[0] += out[j];
        }
        if (a.set_g >= 0) count(2, i, out);
        if (a.dgate && a.dgc && c < cols) {             // a value of its own for each of the row
          if (DT == MOE_T_F32 || a.dgate_f32) store8<MOE_T_F32>((float*)a.dgate + t * a.dgr, c, cols, out);
          else store8<DT>((TD*)a.dgate + t * a.dgr, c, cols, out);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) out[j] = ry * (v.d[j] * v.k[j] * v.w[j] - v.x[j] * mean);
        if (c < cols) store8<DT>((TD*)a.dy + t * a.lddy, c, cols, out);
      }
      if (a.dr && c < cols) {
#pragma unroll
        for (int j = 0; j < 8; ++j) out[j] = v.d[j] * a.alpha;
        store8<RT>((TR*)a.dr + t * a.lddr, c, cols, out);
      }
    });
    if (row_sum_of_gate) {
      row_sums<TPR>(dg, lds);
      if (u0 == 0) {
        if (DT == MOE_T_F32 || a.dgate_f32) ((float*)a.dgate)[t * a.dgr] = dg[0];
        else ((TD*)a.dgate)[t * a.dgr] = Elem<DT>::store(dg[0]);
      }
    }
  }
  if (part >= a.parts) return;
  each([&](int i) __attribute__((always_inline)) {
    const long c = column(i);
    if (c >= cols) return;
    const int set[3] = {a.set_w, a.set_w2, a.set_g};
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      if (set[k] < 0) continue;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (WIDE) v[j] = lds_sums[k * MAX_BWD_COLS + c + j];
        else v[j] = sums[k][i][j];
      }
      store8<MOE_T_F32>(a.part + ((int64_t)set[k] * a.parts + part) * cols, c, cols, v);
    }
  });
}

// Column sums over the parts: 64 columns to a workgroup, its 16 waves every
// 16th part, joined in wave order.
struct JoinArgs {
  const float* part;
  int parts, cols;
  void* to[3];
  int type[3];
};

__global__ void __launch_bounds__(1024)
join_kernel(JoinArgs a) {
  __shared__ float lds[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane, set = blockIdx.y;
  const float* p = a.part + (int64_t)set * a.parts * a.cols;
  float s = 0.0f;
  if (c < a.cols)
    for (int i = wave; i < a.parts; i += 16) s += p[(int64_t)i * a.cols + c];
  lds[wave][lane] = s;
  __syncthreads();
  if (wave || c >= a.cols) return;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) s += lds[i][lane];
  if (a.type[set] == MOE_T_F32) ((float*)a.to[set])[c] = s;
  else if (a.type[set] == MOE_T_BF16) ((uint16_t*)a.to[set])[c] = Elem<MOE_T_BF16>::store(s);
  else ((uint16_t*)a.to[set])[c] = Elem<MOE_T_F16>::store(s);
}

// Threads of a row and units each holds; f(threads, units).  2^25 bf16 values
// with residual and next norm, us: 512 columns by a wave 53, by 256 threads 146;
// 1024 by a wave 50, by 256 threads 83; 4096 by 256 threads 50, by 1024 89.
template <typename F>
int by_width(int64_t cols, F f) {
  typedef std::integral_constant<int, 1> One;
  typedef std::integral_constant<int, 2> Two;
  typedef std::integral_constant<int, 64> Wave;
  typedef std::integral_constant<int, 256> Four;
  typedef std::integral_constant<int, 1024> All;
  if (cols <= 512) return f(Wave(), One());
  if (cols <= 1024) return f(Wave(), Two());
  if (cols <= 2048) return f(Four(), One());
  if (cols <= 4096) return f(Four(), Two());
  if (cols <= 8192) return f(All(), One());
  return f(All(), Two());
}

template <typename F>
int by_types(int dt, int rt, F f) {
  typedef std::integral_constant<int, MOE_T_BF16> BF;
  typedef std::integral_constant<int, MOE_T_F16> HF;
  typedef std::integral_constant<int, MOE_T_F32> F32;
  if (rt == MOE_T_F32)
    return dt == MOE_T_BF16 ? f(BF(), F32()) : dt == MOE_T_F16 ? f(HF(), F32()) : f(F32(), F32());
  return dt == MOE_T_BF16 ? f(BF(), BF()) : f(HF(), HF());
}

// The same for the backward pass (threads of a row, units held).  2^25 bf16
// values, all gradients, us: 512 columns by a wave 124, by 256 threads 309; 1024
// by a wave 157, by 256 threads 172; 4096 held 110, read twice 180; 8192 read
// twice 152 (held, registers spill).
template <typename F>
int by_bwd_width(int64_t cols, F f) {
  typedef std::integral_constant<int, 1> One;
  if (cols <= 512) return f(std::integral_constant<int, 64>(), One());
  if (cols <= 1024) return f(std::integral_constant<int, 64>(), std::integral_constant<int, 2>());
  if (cols <= 2048) return f(std::integral_constant<int, 256>(), One());
  if (cols <= 4096) return f(std::integral_constant<int, 512>(), One());
  return f(std::integral_constant<int, 512>(), std::integral_constant<int, 0>());
}

// Rows the workgroups of the backward pass take in turn, and the waves or
// workgroups whose column sums are joined: as many as the card holds at once.
// Twice as many take 172 us in place of 124 (512 columns), 122 of 108 (2048), 119
// of 110 (4096) for 2^25 values; half of them 143 (512) and 156 (2048).
int64_t bwd_parts(int64_t T, int64_t cols) {
  const int64_t at_once = cols <= 1024 ? 2048 : cols <= 2048 ? 512 : 256;
  return std::max<int64_t>(std::min(T, at_once), 1);
}

int check_types(int dtype, int rtype, int wtype, bool gate, int gtype) {
  if (!elem_bytes(dtype) || !elem_bytes(rtype)) return bad(MOE_E_INVAL, "unknown type");
  if (rtype != dtype && rtype != MOE_T_F32)
    return bad(MOE_E_INVAL, "the residual has the block's type or is fp32");
  if (wtype != dtype && wtype != MOE_T_F32) return bad(MOE_E_INVAL, "weights have the block's type or are fp32");
  if (gate && gtype != dtype && gtype != MOE_T_F32) return bad(MOE_E_INVAL, "the gate has the block's type or is fp32");
  return MOE_OK;
}

int check_size(int64_t T, int64_t cols) {
  if (T < 0 || T > I32_MAX) return bad(MOE_E_INVAL, "rows outside [0, 2^31)");
  if (cols < 1) return bad(MOE_E_INVAL, "need cols >= 1");
  if (cols > MAX_COLS) return bad(MOE_E_UNSUPPORTED, "rows wider than 16384");
  if ((cols > 4096 ? 4 * T : cols > 1024 ? T : (T + 3) / 4) > MAX_BLOCKS) return bad(MOE_E_UNSUPPORTED, "too many rows");
  return MOE_OK;
}

// The memory of a gate (or its gradient) of the given strides.
int check_gate(int64_t gr, int64_t gc, int64_t cols) {
  if (gc != 0 && gc != 1) return bad(MOE_E_INVAL, "a gate's column stride is 0 or 1");
  if (gr < 0 || (gc && gr && gr < cols)) return bad(MOE_E_INVAL, "gate rows overlap");
  if (!gc && !gr) return bad(MOE_E_INVAL, "a gate has a value per row or per column at least");
  return MOE_OK;
}

Span gate_span(const void* p, int64_t T, int64_t cols, int64_t gr, int64_t gc, int b) {
  return row_span(p, gr ? T : 1, gc ? cols : 1, gr ? gr : cols, b);
}

}  // namespace

extern "C" {

int moe_norm(int dtype, const void* y, int64_t ldy, int rtype, const void* residual, int64_t ldr, float alpha,
             int wtype, const void* weight, int gtype, const void* gate, int64_t gate_row, int64_t gate_col, void* h,
             int64_t ldh, const void* next_weight, void* next, int64_t ldn, float* next_scales, int64_t T,
             int64_t cols, float eps, float next_eps, void* stream) {
  int rc = check_types(dtype, rtype, wtype, gate != nullptr, gtype);
  if (rc || (rc = check_size(T, cols))) return rc;
  const int b = elem_bytes(dtype), br = elem_bytes(rtype), bw = elem_bytes(wtype), bg = gate ? elem_bytes(gtype) : 0;
  if ((y && ldy < cols) || (residual && ldr < cols) || (h && ldh < cols) || (next && ldn < cols))
    return bad(MOE_E_INVAL, "row stride smaller than cols");
  if (gate && (rc = check_gate(gate_row, gate_col, cols))) return rc;
  if (T && !y && (weight || gate)) return bad(MOE_E_INVAL, "weight and gate belong to y");
  if (!(eps >= 0.0f) || !(next_eps >= 0.0f)) return bad(MOE_E_INVAL, "eps is not negative");
  const int64_t G = (cols + 127) / 128;
  if (next_scales && (ldn < 128 * G || ldn % 8 || (uintptr_t)next % 8))
    return bad(MOE_E_INVAL, "codes: whole groups, rows on 8 bytes");
  if (T == 0) return MOE_OK;
  if ((!y && !residual) || (!h && !next) || (next && !next_weight) || (next_scales && !next))
    return bad(MOE_E_INVAL, "null argument");
  const bool in_place = h == residual && ldh == ldr;
  if (outputs_shared({row_span(h, T, cols, ldh, br),
                      next_scales ? row_span(next, T, 128 * G, ldn, 1) : row_span(next, T, cols, ldn, b),
                      span(next_scales, G * T * 4)},
                     {row_span(y, T, cols, ldy, b), row_span(in_place ? nullptr : residual, T, cols, ldr, br),
                      span(weight, cols * bw), gate_span(gate, T, cols, gate_row, gate_col, bg),
                      span(next_weight, cols * bw)}) ||
      (in_place && next &&
       meet(next_scales ? row_span(next, T, 128 * G, ldn, 1) : row_span(next, T, cols, ldn, b),
            row_span(residual, T, cols, ldr, br))))
    return shared();
  const NormArgs a{y, ldy, residual, ldr, alpha, weight, gate, gate_row, gate_col, h, ldh, next_weight, next, ldn,
                   next_scales, T, (int)cols, eps, next_eps, wtype == MOE_T_F32, gtype == MOE_T_F32};
  const hipStream_t s = (hipStream_t)stream;
  return by_types(dtype, rtype, [&](auto d, auto r) {
    return by_width(cols, [&](auto tpr, auto nv) {
      const int64_t blocks = tpr.value == 64 ? (T + 3) / 4 : T;
      const unsigned threads = tpr.value == 64 ? 256 : tpr.value;
      if (cols % 8 == 0)
        norm_kernel<d.value, r.value, tpr.value, nv.value, true><<<(unsigned)blocks, threads, 0, s>>>(a);
      else
        norm_kernel<d.value, r.value, tpr.value, nv.value, false><<<(unsigned)blocks, threads, 0, s>>>(a);
      return launched();
    });
  });
}

size_t moe_norm_backward_workspace_bytes(int64_t T, int64_t cols) {
  if (T < 0 || T > I32_MAX || cols < 1 || cols > MAX_BWD_COLS) return 0;
  return (size_t)(3 * bwd_parts(T, cols) * cols * 4);
}

int moe_norm_backward(int dtype, int rtype, const void* dh, int64_t lddh, const void* y, int64_t ldy, float alpha,
                      int wtype, const void* weight, int gtype, const void* gate, int64_t gate_row, int64_t gate_col,
                      const void* dnext, int64_t lddn, const void* h, int64_t ldh, const void* next_weight, void* dy,
                      int64_t lddy, void* dr, int64_t lddr, float* dweight, int dgtype, void* dgate,
                      int64_t dgate_row, int64_t dgate_col, float* dnext_weight, int64_t T, int64_t cols, float eps,
                      float next_eps, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_types(dtype, rtype, wtype, gate != nullptr, gtype);
  if (rc || (rc = check_size(T, cols))) return rc;
  if (cols > MAX_BWD_COLS) return bad(MOE_E_UNSUPPORTED, "gradients of rows wider than 8192");
  const int b = elem_bytes(dtype), br = elem_bytes(rtype), bw = elem_bytes(wtype), bg = gate ? elem_bytes(gtype) : 0;
  if ((dh && lddh < cols) || (y && ldy < cols) || (dnext && lddn < cols) || (dnext && ldh < cols) ||
      (dy && lddy < cols) || (dr && lddr < cols))
    return bad(MOE_E_INVAL, "row stride smaller than cols");
  if (gate && (rc = check_gate(gate_row, gate_col, cols))) return rc;
  if (dgate) {
    if (!gate || (dgtype != dtype && dgtype != MOE_T_F32))
      return bad(MOE_E_INVAL, "the gate's gradient has the block's type or is fp32, beside a gate");
    if ((rc = check_gate(dgate_row, dgate_col, cols))) return rc;
    if (!dgate_row != !gate_row || !dgate_col != !gate_col) return bad(MOE_E_INVAL, "the gate's gradient has its shape");
  }
  if (T && !y && (weight || gate || dy)) return bad(MOE_E_INVAL, "weight, gate and dy belong to y");
  if ((dweight && !weight) || (T && dnext_weight && !dnext)) return bad(MOE_E_INVAL, "a weight's gradient without its norm");
  if (!(eps >= 0.0f) || !(next_eps >= 0.0f)) return bad(MOE_E_INVAL, "eps is not negative");
  if (T && ((!dh && !dnext) || (!dy && !dr) || (y && !dy) || (dnext && (!h || !next_weight))))
    return bad(MOE_E_INVAL, "null argument");
  const int64_t parts = bwd_parts(T, cols);
  const bool gate_sum = dgate && !dgate_row;
  JoinArgs j{(const float*)ws, (int)parts, (int)cols, {}, {}};
  int sets = 0, set_w = -1, set_w2 = -1, set_g = -1;
  const auto add = [&](void* to, int type) {
    j.to[sets] = to;
    j.type[sets] = type;
    return sets++;
  };
  if (dweight) set_w = add(dweight, MOE_T_F32);
  if (dnext_weight) set_w2 = add(dnext_weight, MOE_T_F32);
  if (gate_sum) set_g = add(dgate, dgtype);
  const size_t need = sets ? moe_norm_backward_workspace_bytes(T, cols) : 0;
  if (need && (!ws || ws_bytes < need))
    return bad(MOE_E_INVAL, "workspace smaller than moe_norm_backward_workspace_bytes");
  if (need && (uintptr_t)ws % 4) return bad(MOE_E_INVAL, "the workspace holds floats: it starts on 4 bytes");
  if (T == 0 && !sets) return MOE_OK;
  const int bd = dgtype == MOE_T_F32 ? 4 : 2;
  if (outputs_shared({row_span(dy, T, cols, lddy, b), row_span(dr, T, cols, lddr, br), span(dweight, cols * 4),
                      gate_span(dgate, T, cols, dgate_row, dgate_col, bd), span(dnext_weight, cols * 4),
                      span(need ? ws : nullptr, (int64_t)need)},
                     {row_span(dh, T, cols, lddh, br), row_span(y, T, cols, ldy, b), span(weight, cols * bw),
                      gate_span(gate, T, cols, gate_row, gate_col, bg), row_span(dnext, T, cols, lddn, b),
                      row_span(dnext ? h : nullptr, T, cols, ldh, br), span(dnext ? next_weight : nullptr, cols * bw)}))
    return shared();
  const NormBwdArgs a{dh, lddh, y, ldy, alpha, weight, gate, gate_row, gate_col, dnext, lddn, h, ldh, next_weight, dy,
                      lddy, dr, lddr, gate_sum ? nullptr : dgate, dgate_row, dgate_col, (float*)ws, set_w, set_w2,
                      set_g, T, (int)cols, (int)parts, eps, next_eps, wtype == MOE_T_F32, gtype == MOE_T_F32,
                      dgtype == MOE_T_F32};
  const hipStream_t s = (hipStream_t)stream;
  if (T == 0) j.parts = 0;                             // sums of nothing: no row's memory is touched
  else rc = by_types(dtype, rtype, [&](auto d, auto r) {
    return by_bwd_width(cols, [&](auto tpr, auto nv) {
      const int64_t blocks = tpr.value == 64 ? (parts + 3) / 4 : parts;
      const unsigned threads = tpr.value == 64 ? 256 : tpr.value;
      constexpr int LDS = nv.value == 0 ? 3 * MAX_BWD_COLS * 4 : 0;
      const auto go = [&](auto kernel) {
        if (LDS) {
          const hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, LDS);
          if (e != hipSuccess) return bad(MOE_E_HIP, hipGetErrorString(e));
        }
        kernel<<<(unsigned)blocks, threads, LDS, s>>>(a);
        return launched();
      };
      return cols % 8 == 0 ? go(norm_bwd_kernel<d.value, r.value, tpr.value, nv.value, true>)
                           : go(norm_bwd_kernel<d.value, r.value, tpr.value, nv.value, false>);
    });
  });
  if (rc || !sets) return rc;
  join_kernel<<<dim3((unsigned)((cols + 63) / 64), (unsigned)sets), 1024, 0, s>>>(j);
  return launched();
}

}  // extern "C"
