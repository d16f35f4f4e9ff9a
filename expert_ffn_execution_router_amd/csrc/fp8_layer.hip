// A whole MoE layer for up to 16 tokens, on E4M3 weights with a scale per
// block of 128 x 128, in two kernels:
//
//   z[t, e] = <x[t], R[e]> + b[e];  top-k, w = softmax of the chosen logits
//   a = silu(x G_e^T) * (x U_e^T)  per (token, chosen expert)
//   out[t] = base[t] + sum_j w[t, j] D_e a
//
// The weights are met by 16-bit activations: codes become bf16 or fp16
// exactly, products are exact, sums fp32.
#include "e4m3.h"
#include "op_host.h"
#include "route_dev.h"

namespace {

constexpr int MAX_T = 16, MAX_TOP = 8, MAX_E = 256, MAX_PAIRS = MAX_T * MAX_TOP;
constexpr int WAVES = 4;
constexpr int ROWS = 16;                 // weight rows of a tile

struct LayerArgs {
  const uint16_t* x;
  int64_t ldx;
  const float* router;
  const float* bias;
  int T, E, k, H, I;
  const uint8_t* gu;                     // [E][2I][H]
  const float* sgu;                      // [E][2I/128][H/128]
  const uint8_t* dn;                     // [E][H][I]
  const float* sdn;                      // [E][H/128][I/128]
  const float* base;
  int64_t ldb;
  void* out;
  int64_t ldo;
  int otype;
  int32_t* ids;
  float* w;
  // workspace
  float* z;                              // [T][E]
  unsigned* ctl;                         // tickets, finished gate/up tiles, finished parts of each down tile
  uint16_t* a;                           // [3][T*k][I]
  float* part;                           // [split][H/ROWS][ROWS * MAX_T]
  int split;
};

template <int XT>
struct Frag;
template <>
struct Frag<MOE_T_BF16> {
  typedef bf16x8_t type;
  static DEV f32x4_t mfma(type a, type b, f32x4_t c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
  template <bool HI>
  static DEV int pair(int w) {
    return __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)w, 1.0f, HI));
  }
};
template <>
struct Frag<MOE_T_F16> {
  typedef f16x8_t type;
  static DEV f32x4_t mfma(type a, type b, f32x4_t c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
  template <bool HI>
  static DEV int pair(int w) {
    return __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((uint32_t)w, 1.0f, HI));
  }
};

// 8 codes as 16-bit values, exactly.
template <int XT>
DEV typename Frag<XT>::type widen(int lo, int hi) {
  typedef Frag<XT> F;
  const i32x4_t v = {F::template pair<false>(lo), F::template pair<true>(lo), F::template pair<false>(hi),
                     F::template pair<true>(hi)};
  return __builtin_bit_cast(typename F::type, v);
}

// One wave per expert and four tokens; clears the counters of the second
// kernel, so that the workspace holds nothing from call to call.
template <int XT>
__global__ void __launch_bounds__(256)
router_kernel(LayerArgs a, int n_ctl) {
  const int lane = threadIdx.x & 63;
  if (blockIdx.y == 0)
    for (int i = blockIdx.x * 256 + threadIdx.x; i < n_ctl; i += gridDim.x * 256) a.ctl[i] = 0;
  const int e = blockIdx.x * 4 + (threadIdx.x >> 6), t0 = blockIdx.y * 4;
  if (e >= a.E) return;
  const float* r = a.router + (int64_t)e * a.H;
  float acc[4] = {};
  for (int c0 = 0; c0 < a.H; c0 += 2048) {
    float4 rv[8];
    uint2 xv[8][4];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const int h = min(c0 + c * 256 + lane * 4, a.H - 4);
      rv[c] = *(const float4*)(r + h);
#pragma unroll
      for (int i = 0; i < 4; ++i) xv[c][i] = *(const uint2*)(a.x + min(t0 + i, a.T - 1) * a.ldx + h);
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      if (c0 + c * 256 + lane * 4 >= a.H) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[i] += Elem<XT>::load((uint16_t)(xv[c][i].x & 0xffffu)) * rv[c].x;
        acc[i] += Elem<XT>::load((uint16_t)(xv[c][i].x >> 16)) * rv[c].y;
        acc[i] += Elem<XT>::load((uint16_t)(xv[c][i].y & 0xffffu)) * rv[c].z;
        acc[i] += Elem<XT>::load((uint16_t)(xv[c][i].y >> 16)) * rv[c].w;
      }
    }
  }
  const float b = a.bias ? a.bias[e] : 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float v = wave_sum(acc[i]);
    if (lane == 0 && t0 + i < a.T) a.z[(t0 + i) * a.E + e] = v + b;
  }
}

struct Routed {                          // LDS
  TopkScratch scratch[WAVES];
  int32_t ids[MAX_PAIRS];
  float w[MAX_PAIRS];
  uint32_t bits[MAX_E];                  // tokens of an expert
  int16_t index[MAX_E];
  int16_t act[MAX_PAIRS];                // chosen experts, ascending
  int16_t pair[MAX_PAIRS][MAX_T];        // pair of (chosen expert, token), -1: none
  int n_act;
  unsigned ticket;
  unsigned last;
  __attribute__((aligned(16))) float red[WAVES][2][64][4];
};

DEV void route_all(const LayerArgs& a, Routed& s) {
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, n = a.T * a.k;
  for (int t = wave; t < a.T; t += WAVES) topk_row(a.z + t * a.E, a.E, a.k, s.ids + t * a.k, s.w + t * a.k, nullptr,
                                                   &s.scratch[wave]);
  for (int i = tid; i < MAX_E; i += 64 * WAVES) s.bits[i] = 0;
  for (int i = tid; i < MAX_PAIRS * MAX_T; i += 64 * WAVES) s.pair[i / MAX_T][i % MAX_T] = -1;
  __syncthreads();
  if (tid < n) atomicOr(&s.bits[s.ids[tid]], 1u << (tid / a.k));
  __syncthreads();
  if (wave == 0) {
    int before = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
      const int e = e0 + lane;
      const uint64_t m = __builtin_amdgcn_ballot_w64(e < a.E && s.bits[min(e, MAX_E - 1)] != 0);
      if ((m >> lane) & 1) {
        const int at = before + __popcll(m & ((1ull << lane) - 1));
        s.act[at] = (int16_t)e;
        s.index[e] = (int16_t)at;
      }
      before += __popcll(m);
    }
    if (lane == 0) s.n_act = before;
  }
  __syncthreads();
  if (tid < n) s.pair[s.index[s.ids[tid]]][tid / a.k] = (int16_t)tid;
  __syncthreads();
}

// Sum over the waves of the tile's values: thread (wave i, lane) gets value i
// of the lane.
template <int NT>
DEV void join_waves(const f32x4_t (&acc)[NT], Routed& s, float (&v)[NT]) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < NT; ++i) *(f32x4_t*)s.red[wave][i][lane] = acc[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    v[i] = 0.0f;
#pragma unroll
    for (int q = 0; q < WAVES; ++q) v[i] += s.red[q][i][lane][wave];
  }
}

// Gate and up rows f0 .. f0+15 of a chosen expert, for all of its tokens.
// The waves share out the groups of 128 inputs; the matrix instruction's
// columns are the tokens.  a is kept as three bf16 parts, which hold fp32's
// bits, as the down product's 16-bit operand.
template <int XT>
DEV void gate_up_tile(const LayerArgs& a, Routed& s, int slot, int f0) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const int e = s.act[slot], G = a.H / 128;
  const bool on = s.pair[slot][lr] >= 0;
  const uint8_t* row = a.gu + ((int64_t)e * 2 * a.I + f0 + lr) * a.H + 16 * lg;
  const int64_t up = (int64_t)a.I * a.H;
  const float* sc = a.sgu + ((int64_t)e * (a.I / 64) + f0 / 128) * G;
  const int64_t sup = (int64_t)(a.I / 128) * G;
  const uint16_t* x = a.x + (on ? lr : 0) * a.ldx + 16 * lg;
  f32x4_t acc[2] = {};
  for (int g = wave; g < G; g += WAVES) {
    f32x4_t part[2] = {};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const i32x4_t wg = ld16_nt(row + g * 128 + 64 * h), wu = ld16_nt(row + up + g * 128 + 64 * h);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        i32x4_t xv = {};
        if (on) xv = ld16(x + g * 128 + 64 * h + 8 * q);
        const auto b = __builtin_bit_cast(typename Frag<XT>::type, xv);
        part[0] = Frag<XT>::mfma(widen<XT>(wg[2 * q], wg[2 * q + 1]), b, part[0]);
        part[1] = Frag<XT>::mfma(widen<XT>(wu[2 * q], wu[2 * q + 1]), b, part[1]);
      }
    }
    acc[0] += part[0] * sc[g];
    acc[1] += part[1] * sc[sup + g];
  }
  float v[2];
  join_waves<2>(acc, s, v);
  const int f = f0 + 4 * lg + wave, pair = s.pair[slot][lr];
  if (pair >= 0) {
    const float h = silu(v[0]) * v[1];
    uint16_t* to = a.a + (int64_t)pair * a.I + f;
    const int64_t plane = (int64_t)a.T * a.k * a.I;
    const uint16_t hi = Elem<MOE_T_BF16>::store(h);
    const float r1 = fabsf(h) < INFINITY ? h - bf16_bits_to_f32(hi) : 0.0f;
    const uint16_t mid = Elem<MOE_T_BF16>::store(r1);
    to[0] = hi;
    to[plane] = mid;
    to[2 * plane] = Elem<MOE_T_BF16>::store(r1 - bf16_bits_to_f32(mid));
  }
}

// Rows n0 .. n0+15 of the down product for every token, over part p of the
// (chosen expert, group) list: sum over experts of w[t, j] D_e a in the order
// of the experts, waves taking entries in turn.
DEV void down_tile(const LayerArgs& a, Routed& s, int tile, int p) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const int G = a.I / 128, n = s.n_act * G, n0 = tile * ROWS;
  const int q0 = (int)((int64_t)n * p / a.split), q1 = (int)((int64_t)n * (p + 1) / a.split);
  const int64_t plane = (int64_t)a.T * a.k * a.I;
  f32x4_t acc[1] = {};
  for (int q = q0 + wave; q < q1; q += WAVES) {
    const int slot = q / G, g = q - slot * G, e = s.act[slot], pair = s.pair[slot][lr];
    const uint8_t* row = a.dn + ((int64_t)e * a.H + n0 + lr) * a.I + g * 128 + 16 * lg;
    const uint16_t* h = a.a + (int64_t)max(pair, 0) * a.I + g * 128 + 16 * lg;
    f32x4_t part = {};
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const i32x4_t w = ld16_nt(row + 64 * u);
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const auto m = widen<MOE_T_BF16>(w[2 * v], w[2 * v + 1]);
#pragma unroll
        for (int c = 0; c < 3; ++c) {
          i32x4_t hv = {};
          if (pair >= 0) hv = ld16(h + c * plane + 64 * u + 8 * v);
          part = Frag<MOE_T_BF16>::mfma(m, __builtin_bit_cast(bf16x8_t, hv), part);
        }
      }
    }
    const float sc = a.sdn[((int64_t)e * (a.H / 128) + n0 / 128) * G + g] * s.w[max(pair, 0)];
    if (pair >= 0) acc[0] += part * sc;
  }
  float v[1];
  join_waves<1>(acc, s, v);
  const int r = n0 + 4 * lg + wave, t = lr;
  float sum = v[0];
  if (a.split > 1) {
    const int64_t tiles = a.H / ROWS;
    a.part[((int64_t)p * tiles + tile) * (ROWS * MAX_T) + threadIdx.x] = sum;
    __syncthreads();
    if (threadIdx.x == 0)
      s.last = __hip_atomic_fetch_add(&a.ctl[2 + tile], 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
               (unsigned)a.split - 1;
    __syncthreads();
    if (!s.last) return;
    sum = 0.0f;                          // the parts in their order, whoever came last
    for (int i = 0; i < a.split; ++i) sum += a.part[((int64_t)i * tiles + tile) * (ROWS * MAX_T) + threadIdx.x];
  }
  if (t >= a.T) return;
  if (a.base) sum += a.base[t * a.ldb + r];
  const int64_t at = t * a.ldo + r;
  if (a.otype == MOE_T_F32) ((float*)a.out)[at] = sum;
  else if (a.otype == MOE_T_BF16) ((uint16_t*)a.out)[at] = Elem<MOE_T_BF16>::store(sum);
  else ((uint16_t*)a.out)[at] = Elem<MOE_T_F16>::store(sum);
}

// Workgroups draw tickets: first the gate/up tiles, then the down tiles.  A
// down tile waits until every gate/up tile is finished.  Those have lower
// tickets, so workgroups that run hold them, and gate/up tiles wait for
// nothing: the wait ends however many workgroups are resident.
template <int XT>
__global__ void __launch_bounds__(64 * WAVES)
layer_kernel(LayerArgs a) {
  __shared__ Routed s;
  const int tid = threadIdx.x;
  unsigned mine = 0;
  if (tid == 0) mine = __hip_atomic_fetch_add(&a.ctl[0], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  route_all(a, s);
  const int tiles_a = a.I / ROWS, tiles_b = a.H / ROWS;
  const unsigned na = (unsigned)(s.n_act * tiles_a), all = na + (unsigned)(tiles_b * a.split);
  bool ready = false;
  for (;;) {
    if (tid == 0) s.ticket = mine;
    __syncthreads();
    const unsigned ticket = s.ticket;
    if (ticket >= all) return;
    if (ticket == 0 && tid < a.T * a.k) {
      a.ids[tid] = s.ids[tid];
      a.w[tid] = s.w[tid];
    }
    if (ticket < na) {
      gate_up_tile<XT>(a, s, (int)(ticket / (unsigned)tiles_a), (int)(ticket % (unsigned)tiles_a) * ROWS);
      __syncthreads();
      if (tid == 0) __hip_atomic_fetch_add(&a.ctl[1], 1u, __ATOMIC_RELEASE, __HIP_MEMORY_SCOPE_AGENT);
    } else {
      if (!ready) {
        if (tid == 0)
          while (__hip_atomic_load(&a.ctl[1], __ATOMIC_ACQUIRE, __HIP_MEMORY_SCOPE_AGENT) < na)
            __builtin_amdgcn_s_sleep(1);
        __syncthreads();
        ready = true;
      }
      down_tile(a, s, (int)((ticket - na) % (unsigned)tiles_b), (int)((ticket - na) / (unsigned)tiles_b));
    }
    if (tid == 0) mine = __hip_atomic_fetch_add(&a.ctl[0], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();                     // red and ticket are free
  }
}

int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

int down_split(int64_t k, int64_t H, int64_t I) {
  // about 1024 down tiles, each with an entry for every wave at least
  const int64_t tiles = H / ROWS, entries = k * (I / 128);
  return (int)std::max<int64_t>(1, std::min<int64_t>({1024 / tiles, entries / WAVES, 8}));
}

bool sizes_ok(int64_t T, int64_t E, int64_t k, int64_t H, int64_t I) {
  return T >= 0 && T <= MAX_T && E >= 1 && E <= MAX_E && k >= 1 && k <= MAX_TOP && k <= E && H >= 128 && H <= 32768 &&
         H % 128 == 0 && I >= 128 && I <= 32768 && I % 128 == 0;
}

struct Layout {
  int64_t z, ctl, a, part, end;
  int n_ctl;
};
Layout layout(int64_t T, int64_t E, int64_t k, int64_t H, int64_t I) {
  Layout l;
  l.n_ctl = (int)(2 + H / ROWS);
  l.z = 0;
  l.ctl = up256(T * E * 4);
  l.a = l.ctl + up256(l.n_ctl * 4);
  l.part = l.a + up256(3 * T * k * I * 2);
  l.end = l.part + down_split(k, H, I) * H * MAX_T * 4;
  return l;
}

}  // namespace

extern "C" {

size_t moe_fp8_layer_workspace_bytes(int64_t T, int64_t E, int64_t k, int64_t H, int64_t I) {
  return sizes_ok(T, E, k, H, I) ? (size_t)layout(T, E, k, H, I).end : 0;
}

int moe_fp8_layer(int xtype, const void* x, int64_t ldx, const float* router, const float* bias, int64_t T, int64_t E,
                  int64_t k, int64_t H, int64_t I, const uint8_t* gate_up, const float* gate_up_scales,
                  const uint8_t* down, const float* down_scales, const float* base, int64_t ldb, int otype, void* out,
                  int64_t ldo, int32_t* ids, float* w, void* ws, size_t ws_bytes, void* stream) {
  if (xtype != MOE_T_BF16 && xtype != MOE_T_F16) return bad(MOE_E_INVAL, "x is bf16 or fp16");
  if (otype != xtype && otype != MOE_T_F32) return bad(MOE_E_INVAL, "out has x's type or is fp32");
  if (T < 0 || k < 1 || E < k || H < 1 || I < 1 || H % 128 || I % 128)
    return bad(MOE_E_INVAL, "need T >= 0, 1 <= k <= E, H and I multiples of 128");
  if (!sizes_ok(T, E, k, H, I)) return bad(MOE_E_UNSUPPORTED, "more than 16 tokens, 256 experts, 8 choices or 32768 columns");
  if (ldx < H || ldx % 8 || ldo < H || (base && ldb < H)) return bad(MOE_E_INVAL, "row strides: at least H, x's a multiple of 8");
  if (T == 0) return MOE_OK;
  if (!x || !router || !gate_up || !gate_up_scales || !down || !down_scales || !out || !ids || !w)
    return bad(MOE_E_INVAL, "null argument");
  if (((uintptr_t)x | (uintptr_t)router | (uintptr_t)gate_up | (uintptr_t)down) % 16)
    return bad(MOE_E_INVAL, "x, router and codes start on 16 bytes");
  const Layout l = layout(T, E, k, H, I);
  if (!ws || ws_bytes < (size_t)l.end) return bad(MOE_E_INVAL, "workspace smaller than moe_fp8_layer_workspace_bytes");
  if ((uintptr_t)ws % 16) return bad(MOE_E_INVAL, "the workspace starts on 16 bytes");
  const int bo = otype == MOE_T_F32 ? 4 : 2;
  if (outputs_shared({row_span(out, T, H, ldo, bo), span(ids, T * k * 4), span(w, T * k * 4), span(ws, l.end)},
                     {row_span(x, T, H, ldx, 2), span(router, E * H * 4), span(bias, E * 4),
                      span(gate_up, E * 2 * I * H), span(gate_up_scales, E * (2 * I / 128) * (H / 128) * 4),
                      span(down, E * H * I), span(down_scales, E * (H / 128) * (I / 128) * 4),
                      row_span(base, T, H, ldb, 4)}))
    return shared();
  uint8_t* p = (uint8_t*)ws;
  const LayerArgs a{(const uint16_t*)x, ldx, router, bias, (int)T, (int)E, (int)k, (int)H, (int)I, gate_up,
                    gate_up_scales, down, down_scales, base, ldb, out, ldo, otype, ids, w, (float*)(p + l.z),
                    (unsigned*)(p + l.ctl), (uint16_t*)(p + l.a), (float*)(p + l.part), down_split(k, H, I)};
  const dim3 rg((unsigned)((E + 3) / 4), (unsigned)((T + 3) / 4));
  const int64_t tiles = std::min(E, T * k) * (I / ROWS) + H / ROWS * a.split;
  const unsigned grid = (unsigned)std::min<int64_t>(tiles, 1024);
  const hipStream_t s = (hipStream_t)stream;
  if (xtype == MOE_T_BF16) {
    router_kernel<MOE_T_BF16><<<rg, 256, 0, s>>>(a, l.n_ctl);
    layer_kernel<MOE_T_BF16><<<grid, 64 * WAVES, 0, s>>>(a);
  } else {
    router_kernel<MOE_T_F16><<<rg, 256, 0, s>>>(a, l.n_ctl);
    layer_kernel<MOE_T_F16><<<grid, 64 * WAVES, 0, s>>>(a);
  }
  return launched();
}

}  // extern "C"
