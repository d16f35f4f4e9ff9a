// Expert dispatch as operators of their own: (token, choice) pairs sorted by
// expert, hidden rows copied to their grouped places and back with weights,
// and the gradients of both and of the gate.
//
//   sort      counts[e] = #{a : id_a = e}, segments of align rows' multiples,
//             pos[a] = offsets[id_a] + #{a' < a : id_a' = id_a}
//   permute   xs[pos[t,j]] = x[t]
//   unpermute out[t] = base[t] + sum_j w[t,j] y[pos[t,j]]
//   backward  dy[pos[t,j]] = w[t,j] dout[t],  dw[t,j] = <dout[t], y[pos[t,j]]>
//   gate      dz[t,e] = sum_{j: id = e} w_j (dw_j - sum_i w_i dw_i)
//
// Every sum is fp32 in a fixed order and every rank is counted, not drawn
// from an atomic, so equal inputs give equal bits.
#include "elem.h"
#include "op_host.h"
#include "route_dev.h"

namespace {

// ---------------------------------------------------------------------------
// sort
// ---------------------------------------------------------------------------
// A block ranks up to SORT_WAVES * 64 * ROUNDS pairs: wave v takes a
// contiguous run of 64 * ROUNDS pairs, 64 at a time, and finds in each round
// the lanes that hold the same expert with one ballot per bit of the expert
// id.  The rank inside the wave's run is the wave's count so far plus the
// matching lanes below; the per-wave counts (LDS, one row of E per wave)
// are then scanned over the waves, the blocks and the experts.
constexpr int SORT_WAVES = 8, SORT_THREADS = SORT_WAVES * 64, SORT_ROUNDS = 4;
constexpr int SORT_SPAN = SORT_THREADS * SORT_ROUNDS;      // pairs per block of a multi-block sort
constexpr int SORT_MAX_E = 1024;

// Ranks of the block's pairs inside their wave's run; cnt (LDS, zeroed
// here): [SORT_WAVES][E] pairs of each expert in each wave's run.
template <int ROUNDS>
DEV void rank_pairs(const int32_t* __restrict__ ids, long p0, long n, int E, int* cnt, int (&e)[ROUNDS],
                    int (&rank)[ROUNDS]) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const long w0 = p0 + (long)wave * 64 * ROUNDS + lane;
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    const long p = w0 + 64 * r;
    const int id = p < n ? ids[p] : -1;
    e[r] = (uint32_t)id < (uint32_t)E ? id : -1;
  }
  for (int i = threadIdx.x; i < SORT_WAVES * E; i += SORT_THREADS) cnt[i] = 0;
  __syncthreads();
  const int nb = 32 - __builtin_clz(E);
  int* mine = cnt + wave * E;
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    uint64_t same = __builtin_amdgcn_ballot_w64(e[r] >= 0);
    if (!same) continue;
    for (int b = 0; b < nb; ++b) {
      const bool on = (e[r] >> b) & 1;
      const uint64_t m = __builtin_amdgcn_ballot_w64(on);
      same &= on ? m : ~m;
    }
    const int below = __popcll(same & ((1ull << lane) - 1ull));
    int before = 0;
    if (e[r] >= 0) before = mine[e[r]];
    rank[r] = before + below;
    // the wave's LDS reads and writes complete in program order
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    if (e[r] >= 0 && below == 0) mine[e[r]] = before + __popcll(same);
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
  }
  __syncthreads();
}

// Exclusive scan of the aligned counts over the experts: thread i holds
// experts 2i and 2i+1 (E <= 2 * SORT_THREADS).  Returns the offsets of the
// two and the end of the last segment.  tmp: SORT_WAVES ints of LDS.
DEV int scan_experts(int c0, int c1, int align, int* tmp, int& o0, int& o1) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int a0 = (c0 + align - 1) / align * align, a1 = (c1 + align - 1) / align * align;
  const int inc = wave_incl_sum(a0 + a1);
  if (lane == 63) tmp[wave] = inc;
  __syncthreads();
  int base = 0, end = 0;
#pragma unroll
  for (int i = 0; i < SORT_WAVES; ++i) {
    if (i < wave) base += tmp[i];
    end += tmp[i];
  }
  o0 = base + inc - a0 - a1;
  o1 = o0 + a0;
  return end;
}

// hist (null: this block holds every pair): per block and expert the pairs
// of the blocks before it, then one row of totals.
template <int ROUNDS>
__global__ void __launch_bounds__(SORT_THREADS)
sort_kernel(const int32_t* __restrict__ ids, long n, int E, int align, long rows, const int32_t* __restrict__ hist,
            int32_t* __restrict__ counts, int32_t* __restrict__ offsets, int32_t* __restrict__ perm,
            int32_t* __restrict__ pos) {
  extern __shared__ int lds[];
  int* cnt = lds;                                  // [SORT_WAVES][E], then first rows
  int* seg = lds + SORT_WAVES * E;                 // [E] end of the rows of expert e, [E] end of its segment
  int* tmp = seg + 2 * E;                          // SORT_WAVES
  const long p0 = (long)blockIdx.x * SORT_THREADS * ROUNDS;
  int e[ROUNDS], rank[ROUNDS];
  rank_pairs<ROUNDS>(ids, p0, n, E, cnt, e, rank);
  int tot[2] = {0, 0}, pre[2] = {0, 0}, off[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int x = 2 * threadIdx.x + q;
    if (x >= E) continue;
    if (hist) {
      pre[q] = hist[(size_t)blockIdx.x * E + x];
      tot[q] = hist[(size_t)gridDim.x * E + x];
    } else {
#pragma unroll
      for (int v = 0; v < SORT_WAVES; ++v) tot[q] += cnt[v * E + x];
    }
  }
  const int end = scan_experts(tot[0], tot[1], align, tmp, off[0], off[1]);
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int x = 2 * threadIdx.x + q;
    if (x >= E) continue;
    int at = off[q] + pre[q];
#pragma unroll
    for (int v = 0; v < SORT_WAVES; ++v) {
      const int c = cnt[v * E + x];
      cnt[v * E + x] = at;
      at += c;
    }
    seg[x] = off[q] + tot[q];
    seg[E + x] = off[q] + (tot[q] + align - 1) / align * align;
    if (blockIdx.x == 0) {
      counts[x] = tot[q];
      offsets[x] = off[q];
      if (x == 0) offsets[E] = end;
    }
  }
  __syncthreads();
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    const long p = p0 + (long)wave * 64 * ROUNDS + 64 * r + lane;
    if (p >= n) continue;
    int at = -1;
    if (e[r] >= 0) {
      at = cnt[wave * E + e[r]] + rank[r];
      perm[at] = (int)p;
    }
    pos[p] = at;
  }
  // padding rows of the segments, one wave per expert; rows behind the last
  if (align > 1)
    for (int x = blockIdx.x * SORT_WAVES + wave; x < E; x += gridDim.x * SORT_WAVES)
      for (int r = seg[x] + lane; r < seg[E + x]; r += 64) perm[r] = -1;
  for (long r = end + (long)blockIdx.x * SORT_THREADS + threadIdx.x; r < rows; r += (long)gridDim.x * SORT_THREADS)
    perm[r] = -2;
}

// Pairs of each expert in each block's span.
__global__ void __launch_bounds__(SORT_THREADS)
sort_hist_kernel(const int32_t* __restrict__ ids, long n, int E, int32_t* __restrict__ hist) {
  extern __shared__ int lds[];
  for (int i = threadIdx.x; i < E; i += SORT_THREADS) lds[i] = 0;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < SORT_ROUNDS; ++r) {
    const long p = (long)blockIdx.x * SORT_SPAN + r * SORT_THREADS + threadIdx.x;
    const int id = p < n ? ids[p] : -1;
    if ((uint32_t)id < (uint32_t)E) atomicAdd(&lds[id], 1);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < E; i += SORT_THREADS) hist[(size_t)blockIdx.x * E + i] = lds[i];
}

// In place: hist[b][e] becomes the pairs of e in blocks before b, row nblk
// the totals.  A workgroup takes 64 experts, its 16 waves consecutive runs of
// blocks.
__global__ void __launch_bounds__(1024)
sort_scan_kernel(int32_t* __restrict__ hist, int nblk, int E) {
  __shared__ int part[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = blockIdx.x * 64 + lane;
  const int per = (nblk + 15) / 16, b0 = min(wave * per, nblk), b1 = min(b0 + per, nblk);
  int s = 0;
  if (e < E)
    for (int b = b0; b < b1; ++b) s += hist[(size_t)b * E + e];
  part[wave][lane] = s;
  __syncthreads();
  if (e >= E) return;
  int at = 0;
  for (int v = 0; v < wave; ++v) at += part[v][lane];
  for (int b = b0; b < b1; ++b) {
    const int c = hist[(size_t)b * E + e];
    hist[(size_t)b * E + e] = at;
    at += c;
  }
  if (wave == 15) hist[(size_t)nblk * E + e] = at;
}

// ---------------------------------------------------------------------------
// rows
// ---------------------------------------------------------------------------
// A row is moved in units of V values (16 bytes of the narrower type), the
// last one starting early where the width does not divide, so that it writes
// some values again, with what they hold; rows narrower than a unit go value
// by value.  Units need no alignment beyond the value's.  tpr threads (a
// power of two up to 256) move a row, 256 / tpr rows to a workgroup; at 256 a
// row's index is the workgroup's, so its places and weights are read by scalar
// loads.  HBM bounds the large ones, beside a large copy's 4.8 TB/s: 16384
// tokens x 8 copied rows of 6144 bf16 391 us (1.81 GB, and 0.2 GB of padding
// in segments of 128: 5.1 TB/s), 8192 x 8 combined rows of 2048 59 us (303 MB,
// nine parts in ten read: 5.1 TB/s), gradients of 4096 x 6 rows of 4096 147 us
// (676 MB in three launches: 4.6 TB/s).  Small ragged ones are bound by
// latency: gradients of 777 x 5 fp32 rows of 1001 in segments of 16 take 20 us
// in three launches (45 MB: 2.2 TB/s), half of it in the first, where a
// padding workgroup waits for one perm entry after the other.
struct RowMap {
  int tpr_log2;
};

template <bool WHOLE>
DEV int row_of(const RowMap m, long& row) {
  if (WHOLE) {
    row = blockIdx.x;
    return threadIdx.x;
  }
  row = ((long)blockIdx.x << (8 - m.tpr_log2)) + (threadIdx.x >> m.tpr_log2);
  return threadIdx.x & ((1 << m.tpr_log2) - 1);
}

constexpr int PAD_ROWS = 16;      // grouped rows a padding workgroup looks over

// The value is in registers here (else each store's branch loads it again).
template <typename T, int V>
DEV void pin(Pack<T, V>& v) {
  if constexpr (sizeof(v) == 16) {
    i32x4_t r;
    __builtin_memcpy(&r, &v, sizeof(v));
    asm volatile("" : "+v"(r));
    __builtin_memcpy(&v, &r, sizeof(v));
  } else {
    asm volatile("" : "+v"(v.v[0]));
  }
}

// Copy of token rows to their grouped places: each token row is read once and
// stored k times.  Workgroups past the tokens zero the padding rows (perm -1).
template <typename T, int V, bool WHOLE>
__global__ void __launch_bounds__(256)
permute_kernel(const T* __restrict__ x, long ldx, const int32_t* __restrict__ pos, long nT, int k,
               const int32_t* __restrict__ perm, long rows, int cols, unsigned tok_blocks, RowMap m,
               T* __restrict__ out, long ldo) {
  if (blockIdx.x >= tok_blocks) {
    const Pack<T, V> zero = {};
    const long r0 = (long)(blockIdx.x - tok_blocks) * PAD_ROWS;
    for (int i = 0; i < PAD_ROWS; ++i) {
      const long r = r0 + i;
      if (r >= rows) return;
      if (perm[r] != -1) continue;
      for (int c = threadIdx.x * V; c < cols; c += 256 * V)
        __builtin_memcpy(out + r * ldo + min(c, cols - V), &zero, sizeof(zero));
    }
    return;
  }
  long t;
  const int u0 = row_of<WHOLE>(m, t);
  if (t >= nT) return;
  for (int j0 = 0; j0 < k; j0 += 8) {
    int p[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j] = j0 + j < k ? pos[t * k + j0 + j] : -1;
    for (int c = u0 * V; c < cols; c += V << m.tpr_log2) {
      const int at = min(c, cols - V);
      Pack<T, V> v;
      __builtin_memcpy(&v, x + t * ldx + at, sizeof(v));
      pin(v);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if ((uint32_t)p[j] < (uint64_t)rows) __builtin_memcpy(out + (long)p[j] * ldo + at, &v, sizeof(v));
    }
  }
}

// A token's places and weights, JB choices from j0 on, without branches: past
// the last choice the last again, unused; a dropped pair reads row 0, unused.
template <int JB>
struct Choices {
  long row[JB];
  float w[JB];
  bool use[JB];
  DEV void load(const int32_t* pos, const float* wt, int j0, int k, long rows) {
#pragma unroll
    for (int j = 0; j < JB; ++j) {
      const int jj = min(j0 + j, k - 1), p = pos[jj];
      w[j] = wt ? wt[jj] : 1.0f;
      use[j] = j0 + j < k && (uint32_t)p < (uint64_t)rows;
      row[j] = use[j] ? p : 0;
    }
  }
};

// Weighted sum of a token's grouped rows in choice order, on top of base
// (fp32, may be null); w null: weights of one.  rows > 0.
template <int DY, int DO, int V, int JB, bool WHOLE>
__global__ void __launch_bounds__(256)
unpermute_kernel(const typename Elem<DY>::type* __restrict__ y, long ldy, long rows, const int32_t* __restrict__ pos,
                 const float* __restrict__ w, const float* base, long ldb, long T, int k, int cols, RowMap m,
                 typename Elem<DO>::type* out, long ldo) {
  long t;
  const int u0 = row_of<WHOLE>(m, t);
  if (t >= T) return;
  for (int c = u0 * V; c < cols; c += V << m.tpr_log2) {
    const int at = min(c, cols - V);
    float acc[V];
    if (base) {
      load_vals<MOE_T_F32, V>(base + t * ldb + at, acc);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    }
    for (int j0 = 0; j0 < k; j0 += JB) {
      Choices<JB> ch;
      ch.load(pos + t * k, w ? w + t * k : nullptr, j0, k, rows);
      float v[JB][V];
#pragma unroll
      for (int j = 0; j < JB; ++j) load_vals<DY, V>(y + ch.row[j] * ldy + at, v[j]);
#pragma unroll
      for (int j = 0; j < JB; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = ch.use[j] ? fmaf(ch.w[j], v[j][i], acc[i]) : acc[i];
    }
    store_vals<DO, V>(out + t * ldo + at, acc);
  }
}

// No grouped rows at all: out = base, or zero.
template <int DO>
__global__ void __launch_bounds__(256)
base_only_kernel(const float* base, long ldb, long n, int cols, typename Elem<DO>::type* out, long ldo) {
  const long i = (long)blockIdx.x * 256 + threadIdx.x, t = i / cols;
  if (t >= n) return;
  const int c = (int)(i - t * cols);
  out[t * ldo + c] = Elem<DO>::store(base ? base[t * ldb + c] : 0.0f);
}

// Gradients of unpermute: a token's dout values stay in registers while the
// token's k rows are read (for dw) and their gradients stored.  dw's sum over
// the row: per thread over its units, then a butterfly over the row's lanes,
// then the row's waves in order.  Workgroups past the tokens zero dy's
// padding rows.  rows > 0.
template <int DY, int DO, int V, int JB, bool WHOLE>
__global__ void __launch_bounds__(256)
unpermute_bwd_kernel(const typename Elem<DO>::type* __restrict__ dout, long ldd,
                     const typename Elem<DY>::type* __restrict__ y, long ldy, const int32_t* __restrict__ perm,
                     long rows, const int32_t* __restrict__ pos, const float* __restrict__ w, long T, int k, int cols,
                     unsigned tok_blocks, RowMap m, typename Elem<DY>::type* __restrict__ dy, long lddy,
                     float* __restrict__ dw) {
  if (blockIdx.x >= tok_blocks) {
    const float zero[V] = {};
    const long r0 = (long)(blockIdx.x - tok_blocks) * PAD_ROWS;
    for (int i = 0; i < PAD_ROWS; ++i) {
      const long r = r0 + i;
      if (r >= rows) return;
      if (perm[r] != -1) continue;
      for (int c = threadIdx.x * V; c < cols; c += 256 * V) store_vals<DY, V>(dy + r * lddy + min(c, cols - V), zero);
    }
    return;
  }
  __shared__ float part[4][JB];
  long t;
  const int u0 = row_of<WHOLE>(m, t);
  const bool live = t < T;
  const int tpr = 1 << m.tpr_log2;
  for (int j0 = 0; j0 < k; j0 += JB) {
    float dot[JB];
#pragma unroll
    for (int j = 0; j < JB; ++j) dot[j] = 0.0f;
    if (live) {
      Choices<JB> ch;
      ch.load(pos + t * k, w + t * k, j0, k, rows);
      for (int c = u0 * V; c < cols; c += V * tpr) {
        const int at = min(c, cols - V), again = c - at;        // values another unit has counted
        float g[V], v[JB][V];
        load_vals<DO, V>(dout + t * ldd + at, g);
#pragma unroll
        for (int j = 0; j < JB; ++j) load_vals<DY, V>(y + ch.row[j] * ldy + at, v[j]);
#pragma unroll
        for (int j = 0; j < JB; ++j) {
          float o[V];
#pragma unroll
          for (int i = 0; i < V; ++i) {
            dot[j] = ch.use[j] && i >= again ? fmaf(g[i], v[j][i], dot[j]) : dot[j];
            o[i] = ch.w[j] * g[i];
          }
          if (ch.use[j]) store_vals<DY, V>(dy + ch.row[j] * lddy + at, o);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < JB; ++j)
      for (int off = min(tpr, 64) >> 1; off >= 1; off >>= 1) dot[j] += __shfl_xor(dot[j], off, 64);
    if (tpr > 64) {                            // rows of two or four waves
      const int wave = threadIdx.x >> 6, wpr = tpr >> 6;
      if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int j = 0; j < JB; ++j) part[wave][j] = dot[j];
      __syncthreads();
      const int j = u0;
      if (live && j < JB && j0 + j < k) {
        float s = 0.0f;
        for (int v = 0; v < wpr; ++v) s += part[(wave & ~(wpr - 1)) + v][j];
        dw[t * k + j0 + j] = s;
      }
      __syncthreads();
    } else if (live && u0 == 0) {
#pragma unroll
      for (int j = 0; j < JB; ++j)
        if (j0 + j < k) dw[t * k + j0 + j] = dot[j];
    }
  }
}

__global__ void __launch_bounds__(256) zero_kernel(float* p, long n) {
  const long i = (long)blockIdx.x * 256 + threadIdx.x;
  if (i < n) p[i] = 0.0f;
}

// One wave per token: lane j holds choice j (k <= 64); every lane then sums
// the choices that name its experts.
__global__ void __launch_bounds__(256)
gate_bwd_kernel(const int32_t* __restrict__ ids, const float* __restrict__ w, const float* __restrict__ dw, long T,
                int k, int E, float* __restrict__ dz, long ldz) {
  const long t = (long)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (t >= T) return;
  int id = -1;
  float wv = 0.0f, dv = 0.0f;
  if (lane < k) {
    id = ids[t * k + lane];
    wv = w[t * k + lane];
    dv = dw[t * k + lane];
  }
  const float g = wv * (dv - wave_sum(wv * dv));
  for (int e = lane; e < E; e += 64) {
    float s = 0.0f;
    for (int j = 0; j < k; ++j) {
      const int ij = __builtin_amdgcn_readlane(id, j);
      const float gj = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(g), j));
      s += ij == e ? gj : 0.0f;
    }
    dz[t * ldz + e] = s;
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// Threads per row for `units` units, and the workgroups for T rows.
RowMap row_map_for(int units, long T, long* blocks) {
  int l = 0;
  while (l < 8 && (1 << l) < units) ++l;
  *blocks = (T + (1 << (8 - l)) - 1) >> (8 - l);
  return RowMap{l};
}

constexpr int MAX_K = 64;

long sort_blocks(long n) { return n <= SORT_SPAN ? 1 : (n + SORT_SPAN - 1) / SORT_SPAN; }

// Sizes come in 64 bits, so that none is cut to 32 before it is checked; what
// passes here fits an int.
int check_rows(int64_t T, int64_t k, int64_t rows, int64_t cols) {
  if (T < 0 || k < 1 || k > MAX_K) return bad(MOE_E_INVAL, "need T >= 0 and 1 <= k <= 64");
  if (T > I32_MAX || T * k > I32_MAX) return bad(MOE_E_UNSUPPORTED, "more than 2^31 - 1 pairs");
  if (rows < 0 || rows > I32_MAX) return bad(MOE_E_INVAL, "rows outside [0, 2^31)");
  if (cols < 1) return bad(MOE_E_INVAL, "need cols >= 1");
  if (cols > 1 << 30) return bad(MOE_E_UNSUPPORTED, "rows wider than 2^30");
  return MOE_OK;
}

// f with compile-time types of the two rows, values per unit (one where a
// row is narrower than a unit, or `single`) and choices in flight together.
template <typename F>
int by_types(int dy, int dout, bool single, int cols, int k, F f) {
  const auto choices = [&](auto a, auto b, auto v) {
    if (k == 1) return f(a, b, v, std::integral_constant<int, 1>());
    if (k == 2) return f(a, b, v, std::integral_constant<int, 2>());
    if (k <= 4) return f(a, b, v, std::integral_constant<int, 4>());
    return f(a, b, v, std::integral_constant<int, 8>());
  };
#define CASE(A, B, W)                                                                                          \
  if (dy == A && dout == B)                                                                                    \
    return single || cols < W                                                                                  \
               ? choices(std::integral_constant<int, A>(), std::integral_constant<int, B>(),                   \
                         std::integral_constant<int, 1>())                                                     \
               : choices(std::integral_constant<int, A>(), std::integral_constant<int, B>(),                   \
                         std::integral_constant<int, W>());
  CASE(MOE_T_BF16, MOE_T_BF16, 8)
  CASE(MOE_T_F16, MOE_T_F16, 8)
  CASE(MOE_T_F32, MOE_T_F32, 4)
  CASE(MOE_T_BF16, MOE_T_F32, 8)
  CASE(MOE_T_F16, MOE_T_F32, 8)
  CASE(MOE_T_F32, MOE_T_BF16, 8)
  CASE(MOE_T_F32, MOE_T_F16, 8)
#undef CASE
  return bad(MOE_E_UNSUPPORTED, "types: equal, or one of the two fp32");
}

}  // namespace

extern "C" {

int64_t moe_sort_rows(int64_t T, int64_t k, int64_t E, int64_t align) {
  if (T < 0 || k < 1 || E < 1 || align < 1) return -1;
  if (T > I32_MAX || k > I32_MAX || E > I32_MAX || align > I32_MAX) return -1;      // sums below fit 64 bits
  const int64_t n = T * k;
  return n + (n < E ? n : E) * (align - 1);
}

size_t moe_sort_workspace_bytes(int64_t T, int64_t k, int64_t E) {
  if (T < 0 || k < 1 || E < 1 || T > I32_MAX || k > I32_MAX || E > I32_MAX) return 0;
  const long nb = sort_blocks(T * k);
  return nb == 1 ? 0 : (size_t)(nb + 1) * E * 4;
}

int moe_sort(const int32_t* ids, int64_t T, int64_t k, int64_t E, int64_t align, int32_t* counts, int32_t* offsets,
             int32_t* perm, int64_t rows, int32_t* pos, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_rows(T, k, rows, 1);
  if (rc) return rc;
  if (E < 1 || E > SORT_MAX_E || align < 1 || align > I32_MAX)
    return bad(MOE_E_INVAL, "need 1 <= E <= 1024 and 1 <= align < 2^31");
  if (rows < moe_sort_rows(T, k, E, align)) return bad(MOE_E_INVAL, "perm holds fewer rows than moe_sort_rows");
  const long n = T * k;
  if (!counts || !offsets || (n && (!ids || !pos)) || (rows && !perm)) return bad(MOE_E_INVAL, "null argument");
  const size_t need = moe_sort_workspace_bytes(T, k, E);
  if (need && (!ws || ws_bytes < need)) return bad(MOE_E_INVAL, "workspace smaller than moe_sort_workspace_bytes");
  if (need && (uintptr_t)ws % 4) return bad(MOE_E_INVAL, "the workspace holds ints: it starts on 4 bytes");
  if (outputs_shared({span(counts, E * 4), span(offsets, (E + 1) * 4), span(perm, rows * 4), span(pos, n * 4),
                      span(ws, (int64_t)need)},
                     {span(ids, n * 4)}))
    return shared();
  const hipStream_t s = (hipStream_t)stream;
  const size_t lds = (size_t)((SORT_WAVES + 2) * E + SORT_WAVES) * 4;
  const long nb = sort_blocks(n);
  if (nb == 1) {
    if (n <= SORT_THREADS)
      sort_kernel<1><<<1, SORT_THREADS, lds, s>>>(ids, n, E, align, rows, nullptr, counts, offsets, perm, pos);
    else
      sort_kernel<SORT_ROUNDS><<<1, SORT_THREADS, lds, s>>>(ids, n, E, align, rows, nullptr, counts, offsets, perm,
                                                            pos);
    return launched();
  }
  int32_t* hist = (int32_t*)ws;
  sort_hist_kernel<<<(unsigned)nb, SORT_THREADS, (size_t)E * 4, s>>>(ids, n, E, hist);
  sort_scan_kernel<<<(unsigned)((E + 63) / 64), 1024, 0, s>>>(hist, (int)nb, E);
  sort_kernel<SORT_ROUNDS><<<(unsigned)nb, SORT_THREADS, lds, s>>>(ids, n, E, align, rows, hist, counts, offsets,
                                                                   perm, pos);
  return launched();
}

int moe_permute(int dtype, const void* x, int64_t ldx, const int32_t* perm, const int32_t* pos, int64_t T,
                int64_t k, int64_t rows, int64_t cols, void* out, int64_t ldo, void* stream) {
  int rc = check_rows(T, k, rows, cols);
  if (rc) return rc;
  const int b = elem_bytes(dtype);
  if (!b) return bad(MOE_E_INVAL, "unknown type");
  if (ldx < cols || ldo < cols) return bad(MOE_E_INVAL, "row stride smaller than cols");
  if (rows == 0) return MOE_OK;
  if (!out || (T && (!x || !pos))) return bad(MOE_E_INVAL, "null argument");
  const long pads = perm ? (rows + PAD_ROWS - 1) / PAD_ROWS : 0;
  const hipStream_t s = (hipStream_t)stream;
  const int V = cols < 16 / b ? 1 : 16 / b;
  long blocks;
  const RowMap m = row_map_for((cols + V - 1) / V, T, &blocks);
  if (blocks + pads > MAX_BLOCKS) return bad(MOE_E_UNSUPPORTED, "too many rows");
  if (blocks + pads == 0) return MOE_OK;
  if (outputs_shared({row_span(out, rows, cols, ldo, b)},
                     {row_span(x, T, cols, ldx, b), span(perm, rows * 4), span(pos, T * k * 4)}))
    return shared();
#define GO(U, V, W)                                                                                               \
  permute_kernel<U, V, W><<<(unsigned)(blocks + pads), 256, 0, s>>>((const U*)x, ldx, pos, T, k, perm, rows, cols, \
                                                                    (unsigned)blocks, m, (U*)out, ldo)
  if (b == 4) {
    if (V == 1) GO(uint32_t, 1, false);
    else if (m.tpr_log2 == 8) GO(uint32_t, 4, true);
    else GO(uint32_t, 4, false);
  } else {
    if (V == 1) GO(uint16_t, 1, false);
    else if (m.tpr_log2 == 8) GO(uint16_t, 8, true);
    else GO(uint16_t, 8, false);
  }
#undef GO
  return launched();
}

int moe_unpermute(int ytype, const void* y, int64_t ldy, int64_t rows, const int32_t* pos, const float* w,
                  const float* base, int64_t ldb, int64_t T, int64_t k, int64_t cols, int otype, void* out,
                  int64_t ldo, void* stream) {
  int rc = check_rows(T, k, rows, cols);
  if (rc) return rc;
  const int by = elem_bytes(ytype), bo = elem_bytes(otype);
  if (!by || !bo) return bad(MOE_E_INVAL, "unknown type");
  if (ldy < cols || ldo < cols || (base && ldb < cols)) return bad(MOE_E_INVAL, "row stride smaller than cols");
  if (T == 0) return MOE_OK;
  if ((rows && !y) || !pos || !out) return bad(MOE_E_INVAL, "null argument");
  if (base == out && (otype != MOE_T_F32 || ldb != ldo)) return bad(MOE_E_INVAL, "base is out: fp32, of one stride");
  if (rows == 0 && ((long)T * cols + 255) / 256 > MAX_BLOCKS) return bad(MOE_E_UNSUPPORTED, "too many values");
  const hipStream_t s = (hipStream_t)stream;
  // in place a value may not be read and written twice
  const bool single = base == out && cols % 8 != 0;
  const bool clash = outputs_shared({row_span(out, T, cols, ldo, bo)},
                                    {row_span(y, rows, cols, ldy, by), span(pos, T * k * 4), span(w, T * k * 4),
                                     row_span(base == out ? nullptr : base, T, cols, ldb, 4)});
  return by_types(ytype, otype, single, cols, k, [&](auto a, auto o, auto v, auto jb) {
    typedef typename Elem<a.value>::type TY;
    typedef typename Elem<o.value>::type TO;
    if (rows == 0) {
      if (clash) return shared();
      base_only_kernel<o.value><<<(unsigned)(((long)T * cols + 255) / 256), 256, 0, s>>>(base, ldb, T, cols, (TO*)out,
                                                                                       ldo);
      return launched();
    }
    long blocks;
    const RowMap m = row_map_for((cols + v.value - 1) / v.value, T, &blocks);
    if (blocks > MAX_BLOCKS) return bad(MOE_E_UNSUPPORTED, "too many rows");
    if (clash) return shared();
    if (m.tpr_log2 == 8 && v.value > 1)
      unpermute_kernel<a.value, o.value, v.value, jb.value, true><<<(unsigned)blocks, 256, 0, s>>>(
          (const TY*)y, ldy, rows, pos, w, base, ldb, T, k, cols, m, (TO*)out, ldo);
    else
      unpermute_kernel<a.value, o.value, v.value, jb.value, false><<<(unsigned)blocks, 256, 0, s>>>(
          (const TY*)y, ldy, rows, pos, w, base, ldb, T, k, cols, m, (TO*)out, ldo);
    return launched();
  });
}

int moe_unpermute_backward(int otype, const void* dout, int64_t ldd, int ytype, const void* y, int64_t ldy,
                           const int32_t* perm, int64_t rows, const int32_t* pos, const float* w, int64_t T,
                           int64_t k, int64_t cols, void* dy, int64_t lddy, float* dw, void* stream) {
  int rc = check_rows(T, k, rows, cols);
  if (rc) return rc;
  const int by = elem_bytes(ytype), bo = elem_bytes(otype);
  if (!by || !bo) return bad(MOE_E_INVAL, "unknown type");
  if (ldd < cols || ldy < cols || lddy < cols) return bad(MOE_E_INVAL, "row stride smaller than cols");
  if (T == 0 && (rows == 0 || !perm)) return MOE_OK;
  if ((T && (!dout || !pos || !w || !dw)) || (rows && (!y || !dy))) return bad(MOE_E_INVAL, "null argument");
  const hipStream_t s = (hipStream_t)stream;
  const bool clash = outputs_shared({row_span(dy, rows, cols, lddy, by), span(dw, T * k * 4)},
                                    {row_span(dout, T, cols, ldd, bo), row_span(y, rows, cols, ldy, by),
                                     span(perm, rows * 4), span(pos, T * k * 4), span(w, T * k * 4)});
  return by_types(ytype, otype, false, cols, k, [&](auto a, auto o, auto v, auto jb) {
    typedef typename Elem<a.value>::type TY;
    typedef typename Elem<o.value>::type TO;
    if (rows == 0) {
      if (clash) return shared();
      zero_kernel<<<(unsigned)(((long)T * k + 255) / 256), 256, 0, s>>>(dw, (long)T * k);
      return launched();
    }
    long blocks;
    const RowMap m = row_map_for((cols + v.value - 1) / v.value, T, &blocks);
    const long pads = perm ? (rows + PAD_ROWS - 1) / PAD_ROWS : 0;
    if (blocks + pads > MAX_BLOCKS) return bad(MOE_E_UNSUPPORTED, "too many rows");
    if (clash) return shared();
    if (m.tpr_log2 == 8 && v.value > 1)
      unpermute_bwd_kernel<a.value, o.value, v.value, jb.value, true><<<(unsigned)(blocks + pads), 256, 0, s>>>(
          (const TO*)dout, ldd, (const TY*)y, ldy, perm, rows, pos, w, T, k, cols, (unsigned)blocks, m, (TY*)dy, lddy,
          dw);
    else
      unpermute_bwd_kernel<a.value, o.value, v.value, jb.value, false><<<(unsigned)(blocks + pads), 256, 0, s>>>(
          (const TO*)dout, ldd, (const TY*)y, ldy, perm, rows, pos, w, T, k, cols, (unsigned)blocks, m, (TY*)dy, lddy,
          dw);
    return launched();
  });
}

int moe_gate_backward(const int32_t* ids, const float* w, const float* dw, int64_t T, int64_t k, int64_t E, float* dz,
                      int64_t ldz, void* stream) {
  int rc = check_rows(T, k, 0, 1);
  if (rc) return rc;
  if (E > I32_MAX) return bad(MOE_E_UNSUPPORTED, "more than 2^31 - 1 experts");
  if (E < 1 || ldz < E) return bad(MOE_E_INVAL, "need E >= 1 and a row stride of at least E");
  if (T == 0) return MOE_OK;
  if (!ids || !w || !dw || !dz) return bad(MOE_E_INVAL, "null argument");
  if ((T + 3L) / 4 > MAX_BLOCKS) return bad(MOE_E_UNSUPPORTED, "too many tokens");
  if (outputs_shared({row_span(dz, T, E, ldz, 4)}, {span(ids, T * k * 4), span(w, T * k * 4), span(dw, T * k * 4)}))
    return shared();
  gate_bwd_kernel<<<(unsigned)((T + 3L) / 4), 256, 0, (hipStream_t)stream>>>(ids, w, dw, T, k, E, dz, ldz);
  return launched();
}

}  // extern "C"
