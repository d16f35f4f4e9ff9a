// A whole MoE layer for up to 16 tokens, on E4M3 weights with a scale per
// block of 128 x 128, in two kernels:
//
//   z[t, e] = <x[t], R[e]> + b[e];  top-k, w = softmax of the chosen logits
//   a = silu(x G_e^T) * (x U_e^T)  per (token, chosen expert)
//   out[t] = base[t] + sum_j w[t, j] D_e a
//
// The weights are met by 16-bit activations: codes become bf16 or fp16
// exactly, products are exact, sums fp32.
// The chosen experts' bytes are the floor.  One token of 8 experts (2048 x 768,
// 39 MB): 28.7 us, a chain of waits: the router 4.7, the choice 4, gate/up
// weights 8, their hand-over 3, down 7 with its join.  16 tokens of 6 of 256
// (4096 x 2048, 2.1 GB): 465 us, 4.5 TB/s.
#include "e4m3.h"
#include "op_host.h"
#include "route_dev.h"

namespace {

constexpr int MAX_T = 16, MAX_TOP = 8, MAX_E = 256, MAX_PAIRS = MAX_T * MAX_TOP;
constexpr int WAVES = 4;
constexpr int CTL_WORDS = 32 * 65;         // finished gate/up tiles; 64 flags, a line each
constexpr int CHUNK = 5;                 // tokens whose three parts fit 16 columns
constexpr int U = 2;                     // groups whose weights a wave loads together
constexpr int GRID = 3 * 256;            // workgroups the card holds at once
constexpr int ROWS = 16, DOWN_ROWS = 32;  // weight rows of a gate/up and a down tile

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
  unsigned* ctl;                         // Ctl words, then parts come of each down tile, then claimed gate/up tiles
  uint16_t* a;                           // [3][T*k][I]
  float* part;                           // [split][H/DOWN_ROWS][DOWN_ROWS * MAX_T]
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

// A workgroup per expert and four tokens, its waves sharing out the columns;
// clears the counters of the second kernel, so that the workspace holds
// nothing from call to call.
template <int XT>
__global__ void __launch_bounds__(64 * WAVES)
router_kernel(LayerArgs a, int n_ctl) {
  constexpr int STEP = 256 * WAVES;      // columns of a pass of the workgroup
  __shared__ float lds[WAVES][4];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  if (blockIdx.y == 0)
    for (int i = blockIdx.x * 64 * WAVES + tid; i < n_ctl; i += gridDim.x * 64 * WAVES) a.ctl[i] = 0;
  const int e = blockIdx.x, t0 = blockIdx.y * 4;
  const float* r = a.router + (int64_t)e * a.H;
  float acc[4] = {};
  for (int c0 = 0; c0 < a.H; c0 += 4 * STEP) {
    float4 rv[4];
    uint2 xv[4][4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int h = min(c0 + c * STEP + tid * 4, a.H - 4);
      rv[c] = *(const float4*)(r + h);
#pragma unroll
      for (int i = 0; i < 4; ++i) xv[c][i] = *(const uint2*)(a.x + min(t0 + i, a.T - 1) * a.ldx + h);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (c0 + c * STEP + tid * 4 >= a.H) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[i] += Elem<XT>::load((uint16_t)(xv[c][i].x & 0xffffu)) * rv[c].x;
        acc[i] += Elem<XT>::load((uint16_t)(xv[c][i].x >> 16)) * rv[c].y;
        acc[i] += Elem<XT>::load((uint16_t)(xv[c][i].y & 0xffffu)) * rv[c].z;
        acc[i] += Elem<XT>::load((uint16_t)(xv[c][i].y >> 16)) * rv[c].w;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float v = wave_sum(acc[i]);
    if (lane == 0) lds[wave][i] = v;
  }
  __syncthreads();
  if (tid < 4 && t0 + tid < a.T) {
    float v = 0.0f;
#pragma unroll
    for (int q = 0; q < WAVES; ++q) v += lds[q][tid];
    a.z[(t0 + tid) * a.E + e] = v + (a.bias ? a.bias[e] : 0.0f);
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
  int first[MAX_PAIRS];                  // a token of the chosen expert
  int16_t chunk_e[MAX_PAIRS];            // expert and pairs of each chunk of up to five tokens, -1: none
  int16_t chunk_pair[MAX_PAIRS][CHUNK];
  int16_t chunk_at[MAX_PAIRS];           // first chunk of a chosen expert
  int n_act, n_chunks;
  unsigned pick;
  unsigned last;
  union {
    __attribute__((aligned(16))) float red[WAVES][2][64][4];
    float sums[WAVES][DOWN_ROWS * MAX_T];
  };
};

DEV void route_all(const LayerArgs& a, Routed& s) {
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, n = a.T * a.k;
  for (int t = wave; t < a.T; t += WAVES) topk_row(a.z + t * a.E, a.E, a.k, s.ids + t * a.k, s.w + t * a.k, nullptr,
                                                   &s.scratch[wave]);
  for (int i = tid; i < MAX_E; i += 64 * WAVES) s.bits[i] = 0;
  for (int i = tid; i < n * CHUNK; i += 64 * WAVES) s.chunk_pair[i / CHUNK][i % CHUNK] = -1;
  for (int i = tid; i < n * MAX_T / 2; i += 64 * WAVES) ((uint32_t*)s.pair)[i] = 0xffffffffu;
  __syncthreads();
  if (tid < n) atomicOr(&s.bits[s.ids[tid]], 1u << (tid / a.k));
  __syncthreads();
  if (wave == 0) {
    int before = 0, chunks = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
      const int e = e0 + lane;
      const uint32_t bits = e < a.E ? s.bits[e] : 0;
      const uint64_t m = __builtin_amdgcn_ballot_w64(bits != 0);
      const int nc = (__popc(bits) + CHUNK - 1) / CHUNK, sum = wave_incl_sum(nc);
      if (bits) {
        const int at = before + __popcll(m & ((1ull << lane) - 1));
        s.act[at] = (int16_t)e;
        s.index[e] = (int16_t)at;
        s.first[at] = __builtin_ctz(bits);
        s.chunk_at[at] = (int16_t)(chunks + sum - nc);
      }
      before += __popcll(m);
      chunks += __builtin_amdgcn_readlane(sum, 63);
    }
    if (lane == 0) {
      s.n_act = before;
      s.n_chunks = chunks;
    }
  }
  __syncthreads();
  if (tid < n) {
    const int e = s.ids[tid], slot = s.index[e], t = tid / a.k;
    const int rank = __popc(s.bits[e] & ((1u << t) - 1)), c = s.chunk_at[slot] + rank / CHUNK;
    s.pair[slot][t] = (int16_t)tid;
    s.chunk_e[c] = (int16_t)e;           // by each of its tokens
    s.chunk_pair[c][rank % CHUNK] = (int16_t)tid;
  }
  __syncthreads();
}

// What another workgroup of this launch reads is written through to memory
// (agent scope), and published() waits for it: a release fence instead would
// write back an XCD's whole L2 for each tile.
DEV void publish(uint32_t* p, uint32_t v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
DEV void published() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
  wait_vmcnt<0>();
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
  const uint8_t* row = a.gu + ((int64_t)e * 2 * a.I + f0 + lr) * a.H + 16 * lg;
  const int64_t up = (int64_t)a.I * a.H;
  const float* sc = a.sgu + ((int64_t)e * (a.I / 64) + f0 / 128) * G;
  const int64_t sup = (int64_t)(a.I / 128) * G;
  // columns of other tokens repeat one of the expert's, unused
  const uint16_t* x = a.x + (s.pair[slot][lr] >= 0 ? lr : s.first[slot]) * a.ldx + 16 * lg;
  i32x4_t wn[U][2][2];
  const auto load = [&](int g0) {        // past the last group it again, unused
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int g = min(g0 + u * WAVES, G - 1);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        wn[u][0][h] = ld16_nt(row + g * 128 + 64 * h);
        wn[u][1][h] = ld16_nt(row + up + g * 128 + 64 * h);
      }
    }
  };
  load(wave);
  f32x4_t acc[2] = {};
  for (int g0 = wave; g0 < G; g0 += WAVES * U) {
    i32x4_t wc[U][2][2], xv[U][2][2];
    float sg[U], su[U];
    __builtin_memcpy(wc, wn, sizeof(wc));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int g = min(g0 + u * WAVES, G - 1);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < 2; ++q) xv[u][h][q] = ld16(x + g * 128 + 64 * h + 8 * q);
      sg[u] = sc[g];
      su[u] = sc[sup + g];
    }
    if (g0 + WAVES * U < G) load(g0 + WAVES * U);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (g0 + u * WAVES >= G) break;
      f32x4_t part[2] = {};
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const auto b = __builtin_bit_cast(typename Frag<XT>::type, xv[u][h][q]);
#pragma unroll
          for (int m = 0; m < 2; ++m)
            part[m] = Frag<XT>::mfma(widen<XT>(wc[u][m][h][2 * q], wc[u][m][h][2 * q + 1]), b, part[m]);
        }
      acc[0] += part[0] * sg[u];
      acc[1] += part[1] * su[u];
    }
  }
  float v[2];
  join_waves<2>(acc, s, v);
  const float h = silu(v[0]) * v[1];
  uint16_t hi = Elem<MOE_T_BF16>::store(h);
  if ((hi & 0x7fff) == 0x7f80 && fabsf(h) < INFINITY) --hi;      // the largest there is: the others hold the rest
  const float r1 = fabsf(h) < INFINITY ? h - bf16_bits_to_f32(hi) : 0.0f;
  const uint16_t mid = Elem<MOE_T_BF16>::store(r1), low = Elem<MOE_T_BF16>::store(r1 - bf16_bits_to_f32(mid));
  // thread (wave i, lane) has feature 4 lg + i: two neighbours make a word
  uint16_t* parts = (uint16_t*)s.red;    // [3][16 tokens][16 features]
  __syncthreads();
  const int at = lr * 16 + 4 * lg + wave;
  parts[at] = hi;
  parts[256 + at] = mid;
  parts[512 + at] = low;
  __syncthreads();
  for (int i = threadIdx.x; i < 3 * 128; i += 64 * WAVES) {
    const int c = i >> 7, t = (i >> 3) & 15, w = i & 7, to = s.pair[slot][t];
    if (to >= 0)
      publish((uint32_t*)(a.a + ((int64_t)c * a.T * a.k + to) * a.I + f0) + w, ((const uint32_t*)parts)[c * 128 + t * 8 + w]);
  }
}

// Rows n0 .. n0+31 of the down product for every token, over part p of the
// (chunk, group) list, a chunk being up to five tokens of a chosen expert: the
// three parts of a are columns of one matrix instruction (3 token + part).
// Waves take entries in turn; a chunk's sums, times w[t, j], go to the wave's
// token sums in LDS when its next chunk begins.  wait() returns once a is
// there; the first weights are on their way by then.  a's loads go out before
// the next weights', as loads are waited for in their order.
template <typename F>
DEV void down_tile(const LayerArgs& a, Routed& s, int tile, int p, F wait) {
  constexpr int NT = DOWN_ROWS / 16;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const int G = a.I / 128, n = s.n_chunks * G, n0 = tile * DOWN_ROWS;
  const int q0 = (int)((int64_t)n * p / a.split), q1 = (int)((int64_t)n * (p + 1) / a.split);
  const int col = min(lr / 3, CHUNK - 1), part_of = lr < 3 * CHUNK ? lr % 3 : 0;
  const int64_t plane = (int64_t)a.T * a.k * a.I;
  const uint8_t* rows = a.dn + (int64_t)(n0 + lr) * a.I + 16 * lg;
  const uint16_t* from = a.a + part_of * plane + 16 * lg;
  const float* scales = a.sdn + (int64_t)(n0 / 128) * G;
  float* const sums = s.sums[wave];      // [row][token]
#pragma unroll
  for (int i = 0; i < DOWN_ROWS * MAX_T / 64; ++i) sums[i * 64 + lane] = 0.0f;
  i32x4_t wn[U][NT][2];
  const auto load = [&](int b0) {        // past the last entry it again, unused
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int q = min(b0 + u * WAVES, max(q1 - 1, 0)), c = q / G, g = q - c * G;
      const uint8_t* row = rows + (int64_t)s.chunk_e[c] * a.H * a.I + g * 128;
#pragma unroll
      for (int m = 0; m < NT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) wn[u][m][h] = ld16_nt(row + (int64_t)(16 * m) * a.I + 64 * h);
    }
  };
  load(q0 + wave);
  wait();
  f32x4_t acc[NT] = {};
  int chunk = -1;
  const auto flush = [&] {
    if (chunk < 0) return;
    const int pair = s.chunk_pair[chunk][col];
    const float w = s.w[max(pair, 0)];
#pragma unroll
    for (int m = 0; m < NT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) {      // smallest part first
        const float mid = __shfl(acc[m][i], lane + 1, 64), low = __shfl(acc[m][i], lane + 2, 64);
        const float v = ((low + mid) + acc[m][i]) * w;
        if (pair >= 0 && lr < 3 * CHUNK && part_of == 0)
          sums[(16 * m + 4 * lg + i) * MAX_T + pair / a.k] += v;
        acc[m][i] = 0.0f;
      }
  };
  for (int b0 = q0 + wave; b0 < q1; b0 += WAVES * U) {
    i32x4_t wc[U][NT][2], hv[U][2][2];
    float sc[U];
    __builtin_memcpy(wc, wn, sizeof(wc));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int q = min(b0 + u * WAVES, q1 - 1), c = q / G, g = q - c * G, pair = s.chunk_pair[c][col];
      // columns of no token repeat the first, unused
      const uint16_t* h = from + (int64_t)(pair >= 0 ? pair : s.chunk_pair[c][0]) * a.I + g * 128;
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int v = 0; v < 2; ++v) hv[u][x][v] = ld16(h + 64 * x + 8 * v);
      sc[u] = scales[(int64_t)s.chunk_e[c] * (a.H / 128) * G + g];
    }
    if (b0 + WAVES * U < q1) load(b0 + WAVES * U);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (b0 + u * WAVES >= q1) break;
      const int c = (b0 + u * WAVES) / G;
      if (c != chunk) {
        flush();
        chunk = c;
      }
      f32x4_t part[NT] = {};
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int v = 0; v < 2; ++v)
#pragma unroll
          for (int m = 0; m < NT; ++m)
            part[m] = Frag<MOE_T_BF16>::mfma(widen<MOE_T_BF16>(wc[u][m][x][2 * v], wc[u][m][x][2 * v + 1]),
                                             __builtin_bit_cast(bf16x8_t, hv[u][x][v]), part[m]);
#pragma unroll
      for (int m = 0; m < NT; ++m) acc[m] += part[m] * sc[u];
    }
  }
  flush();
  __syncthreads();
  // value i * 256 + thread: row, token
  constexpr int NV = DOWN_ROWS * MAX_T / (64 * WAVES);
  const int64_t tiles = a.H / DOWN_ROWS;
  float v[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    v[i] = 0.0f;
#pragma unroll
    for (int q = 0; q < WAVES; ++q) v[i] += s.sums[q][i * 64 * WAVES + threadIdx.x];
  }
  if (a.split > 1) {
    float* mine = a.part + ((int64_t)p * tiles + tile) * (DOWN_ROWS * MAX_T) + threadIdx.x;
#pragma unroll
    for (int i = 0; i < NV; ++i) publish((uint32_t*)mine + i * 64 * WAVES, __float_as_uint(v[i]));
    published();
    if (threadIdx.x == 0)
      s.last = __hip_atomic_fetch_add(&a.ctl[CTL_WORDS + tile], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
               (unsigned)a.split - 1;
    __syncthreads();
    if (!s.last) return;
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = 0.0f;
    for (int q = 0; q < a.split; ++q)    // the parts in their order, whoever came last
#pragma unroll
      for (int i = 0; i < NV; ++i)
        v[i] += __hip_atomic_load(a.part + ((int64_t)q * tiles + tile) * (DOWN_ROWS * MAX_T) + threadIdx.x + i * 64 * WAVES,
                                  __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = i * 64 * WAVES + threadIdx.x, r = n0 + at / MAX_T, t = at % MAX_T;
    if (t >= a.T) continue;
    float sum = v[i];
    if (a.base) sum += a.base[t * a.ldb + r];
    const int64_t to = t * a.ldo + r;
    if (a.otype == MOE_T_F32) ((float*)a.out)[to] = sum;
    else if (a.otype == MOE_T_BF16) ((uint16_t*)a.out)[to] = Elem<MOE_T_BF16>::store(sum);
    else ((uint16_t*)a.out)[to] = Elem<MOE_T_F16>::store(sum);
  }
}

// Workgroups take gate/up tiles blockIdx, + gridDim, .. and then down tiles from
// the last workgroup backwards, so that with few tokens those without a gate/up
// tile have the down weights on their way while the others work.  A down tile waits until every gate/up tile is finished, however
// few workgroups are resident: each gate/up tile is claimed before it is begun,
// and one with a down tile takes what is left unclaimed before it waits.
// So what it waits for is held by running workgroups, which wait for nothing
// until they have finished it.  The last one to finish raises the flags: each
// is polled by few workgroups, and the counter by none.
template <int XT>
__global__ void __launch_bounds__(64 * WAVES, 3)
layer_kernel(LayerArgs a) {
  __shared__ Routed s;
  const int tid = threadIdx.x;
  const int tiles_a = a.I / ROWS, tiles_b = a.H / DOWN_ROWS;
  unsigned* const claimed = a.ctl + CTL_WORDS + tiles_b;
  const int bound = min(a.E, a.T * a.k) * tiles_a;
  unsigned taken = 0;
  const auto claim = [&](int tile) {
    if (tid == 0 && tile < bound)
      taken = __hip_atomic_exchange(&claimed[tile], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  };
  claim(blockIdx.x);
  route_all(a, s);
  const int na = s.n_act * tiles_a;
  if (blockIdx.x == 0 && tid < a.T * a.k) {
    a.ids[tid] = s.ids[tid];
    a.w[tid] = s.w[tid];
  }
  const auto gate_up = [&](int tile) {
    gate_up_tile<XT>(a, s, tile / tiles_a, tile % tiles_a * ROWS);
    published();
    if (tid < 64) {
      unsigned before = 0;
      if (tid == 0) before = __hip_atomic_fetch_add(&a.ctl[0], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (__builtin_amdgcn_readfirstlane(before) == (unsigned)na - 1) publish(&a.ctl[32 * (1 + tid)], 1);
    }
  };
  for (int tile = blockIdx.x; tile < na; tile += gridDim.x) {
    if (tid == 0) s.pick = taken;
    __syncthreads();
    const unsigned mine = s.pick;
    claim(tile + gridDim.x);
    if (mine == 0) gate_up(tile);
    __syncthreads();
  }
  const int d0 = gridDim.x - 1 - blockIdx.x;
  if (d0 >= tiles_b * a.split) return;
  for (;;) {
    if (tid == 0) s.pick = 0xffffffffu;
    __syncthreads();
    unsigned best = 0xffffffffu;         // the first unclaimed one after a place of its own
    const unsigned start = (unsigned)((int64_t)blockIdx.x * na / gridDim.x);
    for (int i = tid; i < na; i += 64 * WAVES) {
      const unsigned at = (start + i) % (unsigned)na;
      if (best == 0xffffffffu && !__hip_atomic_load(&claimed[at], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)) best = i;
    }
    if (best != 0xffffffffu) atomicMin(&s.pick, best);
    __syncthreads();
    if (s.pick == 0xffffffffu) break;
    const int tile = (int)((start + s.pick) % (unsigned)na);
    __syncthreads();
    claim(tile);
    if (tid == 0) s.pick = taken;
    __syncthreads();
    const unsigned mine = s.pick;
    if (mine == 0) gate_up(tile);
    __syncthreads();
  }
  bool ready = false;
  for (int d = d0; d < tiles_b * a.split; d += gridDim.x) {
    down_tile(a, s, d % tiles_b, d / tiles_b, [&] {
      if (ready) return;
      if (tid == 0) {
        while (!__hip_atomic_load(&a.ctl[32 * (1 + blockIdx.x % 64)], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT))
          __builtin_amdgcn_s_sleep(1);
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
      }
      __syncthreads();
      ready = true;
    });
    __syncthreads();                     // red is free
  }
}

int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

// Down tiles for each 32 rows: about 512 in all or, where that leaves at least
// half as many, one for each workgroup without a gate/up tile (one token of 8
// experts, 2048 x 768: 33.3 us with its launches, 34.9 with 512), with an entry
// for every wave at least.
int down_split(int64_t T, int64_t E, int64_t k, int64_t H, int64_t I) {
  const int64_t tiles = H / DOWN_ROWS, entries = k * (I / 128), many = 512 / tiles;
  const int64_t free = (GRID - std::min(E, T * k) * (I / ROWS)) / tiles;
  const int64_t parts = 2 * free >= many ? std::min(free, many) : many;
  return (int)std::max<int64_t>(1, std::min<int64_t>({parts, entries / WAVES, 8}));
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
  l.n_ctl = (int)(CTL_WORDS + H / DOWN_ROWS + std::min(E, T * k) * (I / ROWS));
  l.z = 0;
  l.ctl = up256(T * E * 4);
  l.a = l.ctl + up256(l.n_ctl * 4);
  l.part = l.a + up256(3 * T * k * I * 2);
  l.end = l.part + down_split(T, E, k, H, I) * H * MAX_T * 4;
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
                    (unsigned*)(p + l.ctl), (uint16_t*)(p + l.a), (float*)(p + l.part), down_split(T, E, k, H, I)};
  const dim3 rg((unsigned)E, (unsigned)((T + 3) / 4));
  const int64_t tiles = std::min(E, T * k) * (I / ROWS) + H / DOWN_ROWS * a.split;
  const unsigned grid = (unsigned)std::min<int64_t>(tiles, GRID);
  const hipStream_t s = (hipStream_t)stream;
  if (xtype == MOE_T_BF16) {
    router_kernel<MOE_T_BF16><<<rg, 64 * WAVES, 0, s>>>(a, l.n_ctl);
    layer_kernel<MOE_T_BF16><<<grid, 64 * WAVES, 0, s>>>(a);
  } else {
    router_kernel<MOE_T_F16><<<rg, 64 * WAVES, 0, s>>>(a, l.n_ctl);
    layer_kernel<MOE_T_F16><<<grid, 64 * WAVES, 0, s>>>(a);
  }
  return launched();
}

}  // extern "C"
