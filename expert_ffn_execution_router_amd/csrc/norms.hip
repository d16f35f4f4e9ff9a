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
// A row is read once and held in registers, as units of 8 columns: 64, 256 or
// 1024 threads with up to two units each.  All sums are fp32 in a fixed order.
#include "e4m3.h"
#include "op_host.h"

namespace {

constexpr int MAX_COLS = 16384;

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

// Sum over the threads of a row: one wave, or all waves of the workgroup.
template <int TPR>
DEV float row_sum(float v, float* lds) {
  v = wave_sum(v);
  if (TPR == 64) return v;
  __syncthreads();                               // lds is free again
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < TPR / 64; ++i) s += lds[i];
  return s;
}

template <int DT>
DEV void load_param(const void* p, bool f32, long c, long cols, float (&f)[8]) {
  if (DT == MOE_T_F32 || f32) load8<MOE_T_F32>((const float*)p, c, cols, f);
  else load8<DT>((const typename Elem<DT>::type*)p, c, cols, f);
}

// The gate of row t, columns c .. c+7 (zeros past cols).
template <int DT>
DEV void load_gate(const void* p, bool f32, int64_t t, int64_t gr, int64_t gc, long c, long cols, float (&f)[8]) {
  typedef typename Elem<DT>::type T;
  if (gc == 0) {
    const float g = DT == MOE_T_F32 || f32 ? ((const float*)p)[t * gr] : Elem<DT>::load(((const T*)p)[t * gr]);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = g;
  } else if (DT == MOE_T_F32 || f32) {
    load8<MOE_T_F32>((const float*)p + t * gr, c, cols, f);
  } else {
    load8<DT>((const T*)p + t * gr, c, cols, f);
  }
}

template <int DT, int RT, int TPR, int NV>
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
    for (int i = 0; i < NV; ++i) load8<RT>((const TR*)a.r + t * a.ldr, (u0 + i * TPR) * 8, cols, h[i]);
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
    for (int i = 0; i < NV; ++i) load8<DT>((const TD*)a.y + t * a.ldy, (u0 + i * TPR) * 8, cols, y[i]);
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
        load_param<DT>(a.w, a.w_f32, c, cols, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[i][j] = y[i][j] * rs * w[j];
      }
      if (a.gate) {
        float g[8];
        load_gate<DT>(a.gate, a.gate_f32, t, a.gr, a.gc, c, cols, g);
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
    load_param<DT>(a.w2, a.w_f32, c, cols, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) h[i][j] = c + j < cols ? h[i][j] * rs * w[j] : 0.0f;
    if (!a.scales) {
      if (c < cols) store8<DT>((TD*)a.next + t * a.ldn, c, cols, h[i]);
      continue;
    }
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, abs_bits(h[i][j]));
    const GroupScale q = group_scale(row16_max(m));
    if (c / 128 * 128 >= cols) continue;             // whole groups: the last one's tail is zeros
    const uint2 v = {codes4(h[i][0], h[i][1], h[i][2], h[i][3], q.inv),
                     codes4(h[i][4], h[i][5], h[i][6], h[i][7], q.inv)};
    *(uint2*)((uint8_t*)a.next + t * a.ldn + c) = v;
    if ((u0 & 15) == 0) a.scales[c / 128 * a.T + t] = q.scale;
  }
}

template <int DT, int RT, int TPR, int NV>
__global__ void __launch_bounds__(TPR == 64 ? 256 : TPR)
norm_bwd_kernel(NormBwdArgs a) {
  typedef typename Elem<DT>::type TD;
  typedef typename Elem<RT>::type TR;
  __shared__ float lds[16];
  const int u0 = TPR == 64 ? threadIdx.x & 63 : threadIdx.x;
  const int part = TPR == 64 ? blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  const int cols = a.cols;
  const float inv_n = 1.0f / (float)cols;
  float sw[NV][8] = {}, sw2[NV][8] = {}, sg[NV][8] = {};
  for (int64_t t = part; t < a.T; t += a.parts) {
    float d[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (a.dh) load8<RT>((const TR*)a.dh + t * a.lddh, (u0 + i * TPR) * 8, cols, d[i]);
      else
#pragma unroll
        for (int j = 0; j < 8; ++j) d[i][j] = 0.0f;
    }
    if (a.dn) {
      float n[NV][8], g[NV][8], s = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        load8<RT>((const TR*)a.h + t * a.ldh, (u0 + i * TPR) * 8, cols, n[i]);
        load8<DT>((const TD*)a.dn + t * a.lddn, (u0 + i * TPR) * 8, cols, g[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) s += n[i][j] * n[i][j];
      }
      const float rs = 1.0f / sqrtf(row_sum<TPR>(s, lds) * inv_n + a.eps2);
      s = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float w[8];
        load_param<DT>(a.w2, a.w_f32, (u0 + i * TPR) * 8, cols, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          n[i][j] *= rs;
          sw2[i][j] += g[i][j] * n[i][j];
          g[i][j] *= w[j];
          s += g[i][j] * n[i][j];
        }
      }
      const float mean = row_sum<TPR>(s, lds) * inv_n;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) d[i][j] += rs * (g[i][j] - n[i][j] * mean);
    }
    if (a.y) {
      float x[NV][8], dv[NV][8], rs = 1.0f, s = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        load8<DT>((const TD*)a.y + t * a.ldy, (u0 + i * TPR) * 8, cols, x[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) s += x[i][j] * x[i][j];
      }
      if (a.w) rs = 1.0f / sqrtf(row_sum<TPR>(s, lds) * inv_n + a.eps);
      float mean = 0.0f, dg = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const long c = (u0 + i * TPR) * 8;
        float w[8], g[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = g[j] = 1.0f;
        if (a.w) load_param<DT>(a.w, a.w_f32, c, cols, w);
        if (a.gate) load_gate<DT>(a.gate, a.gate_f32, t, a.gr, a.gc, c, cols, g);
        float full[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[i][j] *= rs;
          const float e = d[i][j] * x[i][j];
          full[j] = e * w[j];
          dg += full[j];
          sg[i][j] += full[j];
          sw[i][j] += e * g[j];
          dv[i][j] = d[i][j] * g[j] * w[j];
          mean += dv[i][j] * x[i][j];
        }
        if (a.dgate && a.dgc && c < cols) {           // a value of its own for each of the row
          if (DT == MOE_T_F32 || a.dgate_f32) store8<MOE_T_F32>((float*)a.dgate + t * a.dgr, c, cols, full);
          else store8<DT>((TD*)a.dgate + t * a.dgr, c, cols, full);
        }
      }
      mean = a.w ? row_sum<TPR>(mean, lds) * inv_n : 0.0f;
      if (a.dgate && !a.dgc) {
        dg = row_sum<TPR>(dg, lds);
        if (u0 == 0) {
          if (DT == MOE_T_F32 || a.dgate_f32) ((float*)a.dgate)[t * a.dgr] = dg;
          else ((TD*)a.dgate)[t * a.dgr] = Elem<DT>::store(dg);
        }
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const long c = (u0 + i * TPR) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) dv[i][j] = rs * (dv[i][j] - x[i][j] * mean);
        if (c < cols) store8<DT>((TD*)a.dy + t * a.lddy, c, cols, dv[i]);
      }
    }
    if (a.dr) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const long c = (u0 + i * TPR) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) d[i][j] *= a.alpha;
        if (c < cols) store8<RT>((TR*)a.dr + t * a.lddr, c, cols, d[i]);
      }
    }
  }
  if (part >= a.parts) return;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const long c = (u0 + i * TPR) * 8;
    if (c >= cols) continue;
    const auto put = [&](int set, const float (&v)[8]) {
      if (set >= 0) store8<MOE_T_F32>(a.part + ((int64_t)set * a.parts + part) * cols, c, cols, v);
    };
    put(a.set_w, sw[i]);
    put(a.set_w2, sw2[i]);
    put(a.set_g, sg[i]);
  }
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

// Threads of a row and units each holds; f(threads, units).
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

// Rows the workgroups of the backward pass take in turn, and the waves or
// workgroups whose column sums are joined.
int64_t bwd_parts(int64_t T, int64_t cols) {
  const int64_t at_once = cols <= 1024 ? 4096 : cols <= 4096 ? 1024 : 512;
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
  return by_types(dtype, rtype, [&](auto d, auto r) {
    return by_width(cols, [&](auto tpr, auto nv) {
      const int64_t blocks = tpr.value == 64 ? (T + 3) / 4 : T;
      norm_kernel<d.value, r.value, tpr.value, nv.value>
          <<<(unsigned)blocks, tpr.value == 64 ? 256 : tpr.value, 0, (hipStream_t)stream>>>(a);
      return launched();
    });
  });
}

size_t moe_norm_backward_workspace_bytes(int64_t T, int64_t cols) {
  if (T < 0 || T > I32_MAX || cols < 1 || cols > MAX_COLS) return 0;
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
  rc = by_types(dtype, rtype, [&](auto d, auto r) {
    return by_width(cols, [&](auto tpr, auto nv) {
      const int64_t blocks = tpr.value == 64 ? (parts + 3) / 4 : parts;
      norm_bwd_kernel<d.value, r.value, tpr.value, nv.value>
          <<<(unsigned)blocks, tpr.value == 64 ? 256 : tpr.value, 0, s>>>(a);
      return launched();
    });
  });
  if (rc || !sets) return rc;
  join_kernel<<<dim3((unsigned)((cols + 63) / 64), (unsigned)sets), 1024, 0, s>>>(j);
  return launched();
}

}  // extern "C"
