// Attention among the rows of each segment for gfx950: forward and the two
// passes of its VJP.  For query row i, key row j of one segment and a head:
//   u = scale <q_i, k_j>,  t = cap tanh(u / cap)  (t = u without a cap),
//   s = t - slope |p_i - p_j|,  absent unless j < vis_i,
//   lse_i = log sum_j exp(s),  P = exp(s - lse_i),  o_i = sum_j P v_j;
//   vis_i = max(prefix, i + (Lk - Lq) + 1) when causal, else Lk.
// For the cotangent g of o, dP = <g_i, v_j>, delta_i = sum_j P dP = <g_i, o_i>,
//   dS = P (dP - delta_i),  du = dS (1 - (t/cap)^2) scale,
//   q_bar = sum_j du k_j,  k_bar = sum_i du q_i,  v_bar = sum_i P g_i,
//   slope_bar = - sum dS r,  p_bar_i = - sum_heads slope sum_j dS (p_i - p_j) / r.
// A row that sees no key has o = 0, lse = -inf and adds nothing.
//
// Layout.  Every kernel keeps 32 "columns" per wave in registers and walks
// the other axis in tiles of rows through LDS.  The forward and the query
// pass hold query rows as columns and walk keys, the key pass holds key rows
// and walks queries.  The query heads that share a key head are packed into
// one axis (row = i G + head), so that each key row is loaded once for all of
// them and the sums over shared heads need no extra step.  The product
// rows x columns comes out of the 32x32 matrix instruction with a column per
// lane: maxima and sums over rows stay in the lane (plus one exchange between
// the wave's halves), and the same registers are the right-hand operand of
// the second product, whose left-hand side is the row tile read transposed
// (ds_read_b64_tr_b16 for bfloat16, plain reads for fp32).
//
// No atomics: each output has one writer, and the VJP is two passes, which
// repeats the scores (seven products instead of five) but keeps results
// bitwise reproducible.
#pragma once

#include <hip/hip_runtime.h>

#include "fc_attn.h"
#include "fc_types.h"

namespace fc {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

inline constexpr float kLog2e = 1.44269504088896340736f;
inline constexpr float kLn2 = 0.69314718055994530942f;
inline constexpr float kInf = __builtin_huge_valf();

// 16 bytes of a row: the unit of every load, and one step of a product
template <class T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int kChunk = 4;
  using Frag = f32x4;
};
template <>
struct Elem<bf16> {
  static constexpr int kChunk = 8;
  using Frag = bf16x8;
};

// acc[row][col] += A[row][.] B[col][.] over two chunks (one per half wave)
__device__ __forceinline__ f32x16 mma(f32x4 a, f32x4 b, f32x16 c) {
#pragma unroll
  for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i], b[i], c, 0, 0, 0);
  return c;
}
__device__ __forceinline__ f32x16 mma(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Row of register r of the 32x32 result, for the wave's half h.
__device__ __forceinline__ constexpr int acc_row(int r, int h) { return (r / 4) * 8 + h * 4 + r % 4; }

template <class T, int DP>
struct Tile {
  static constexpr int CH = Elem<T>::kChunk;
  using Frag = typename Elem<T>::Frag;
  static constexpr int STEPS = DP / (2 * CH);          // products over d
  static constexpr int DB = (DP + 31) / 32;            // 32-wide blocks of d
  static constexpr int LD = DB * 32 + CH;              // LDS row: 16 bytes of padding spread the banks
  static constexpr int CPR = DP / CH;                  // chunks of a row
  static_assert(DP % (2 * CH) == 0);

  // columns of a wave: lane -> its column's chunk 2 s + h
  static __device__ __forceinline__ void load_cols(const T* row, bool live, int D, int h, Frag (&f)[STEPS]) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int d = (2 * s + h) * CH;
      Frag z = {};
      f[s] = live && d < D ? *reinterpret_cast<const Frag*>(row + d) : z;
    }
  }

  // acc[row][col] = sum_d rows[row][d] cols[col][d] for 32 rows in LDS
  static __device__ __forceinline__ f32x16 dot(const T* rows, const Frag (&cols)[STEPS], int lane) {
    f32x16 c = {};
    const T* p = rows + (lane % 32) * LD + (lane / 32) * CH;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) c = mma(*reinterpret_cast<const Frag*>(p + 2 * s * CH), cols[s], c);
    return c;
  }

  // out[d][col] += sum_row rows[row][d] w[row][col] for 32 rows in LDS
  static __device__ __forceinline__ void outer(const T* rows, const f32x16& w, f32x16 (&out)[DB], int lane) {
    if constexpr (sizeof(T) == 4) {
      const T* p = rows + (lane / 32) * 4 * LD + lane % 32;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const T* pr = p + acc_row(r, 0) * LD;
#pragma unroll
        for (int b = 0; b < DB; ++b)
          out[b] = __builtin_amdgcn_mfma_f32_32x32x2f32(pr[b * 32], w[r], out[b], 0, 0, 0);
      }
    } else {
      // 16 lanes read four rows x 16 columns and get a column each
      const T* p = rows + ((lane / 32) * 4 + (lane % 16) / 4) * LD + ((lane / 16) % 2) * 16 + (lane % 4) * 4;
      typedef __attribute__((address_space(3))) i16x4* lds_ptr;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        bf16x8 wb;   // rounded to bfloat16 as the matrix instruction takes it
#pragma unroll
        for (int i = 0; i < 8; ++i) wb[i] = static_cast<bf16>(w[8 * s + i]);
#pragma unroll
        for (int b = 0; b < DB; ++b) {
          const T* pb = p + s * 16 * LD + b * 32;
          const bf16x4 lo = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(pb)));
          const bf16x4 hi = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(pb + 8 * LD)));
          out[b] = mma(__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7), wb, out[b]);
        }
      }
    }
  }
};

// A tile of ROWS rows on its way from memory to LDS: loaded into registers
// while the tile before is worked on, then stored.
template <class T, int DP, int ROWS, int THREADS>
struct Stage {
  using TL = Tile<T, DP>;
  static constexpr int N = (ROWS * TL::CPR + THREADS - 1) / THREADS;
  f32x4 r[N];

  // row(i) gives the address of tile row i, null for a row of zeros
  template <class F>
  __device__ __forceinline__ void load(int D, F&& row) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = i * THREADS + threadIdx.x;
      const int rr = e / TL::CPR, d = (e % TL::CPR) * TL::CH;
      f32x4 z = {};
      r[i] = z;
      if ((ROWS * TL::CPR % THREADS == 0 || rr < ROWS) && d < D) {
        const T* p = row(rr);
        if (p) r[i] = *reinterpret_cast<const f32x4*>(p + d);
      }
    }
  }
  __device__ __forceinline__ void store(T* lds) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = i * THREADS + threadIdx.x;
      const int rr = e / TL::CPR, d = (e % TL::CPR) * TL::CH;
      if (ROWS * TL::CPR % THREADS == 0 || rr < ROWS) *reinterpret_cast<f32x4*>(lds + rr * TL::LD + d) = r[i];
    }
  }
};

__device__ __forceinline__ float other_half(float x) { return __shfl_xor(x, 32); }

// tanh from one exponential; its error is that of 1 - tanh, a few 2^-24
__device__ __forceinline__ float tanh_fast(float x) {
  return 1.f - 2.f * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(x * (2.f * kLog2e)));
}

// ------------------------------------------------- which work a block has --

struct Work {
  int seg, tile, head, split;   // segment, column tile in it, key head
  int q0, lq, k0, lk, pre;
  bool any;
};

// Tiles of `cols` columns: segment s starts at tile off[s] mul / cols + s,
// which leaves every segment room for its last, partial tile without a scan
// over the segments before it (at most one tile per segment stays empty).
__device__ __forceinline__ int64_t tile_start(const int* off, int s, int mul, int cols) {
  return (off ? (int64_t)off[s] * mul / cols : 0) + s;
}

// The column axis is queries (mul = G) or keys (mul = 1).  All lanes of a
// wave search together, 64 segments per step.
template <bool KEYS>
__device__ __forceinline__ Work find_work(const AttnArgs& a, int cols, int tiles, int splits) {
  Work w{};
  const int units = a.hk * splits;
  int unit, t;
  const int b = blockIdx.x;
  // Blocks go to the eight dies in turn.  A die takes whole (key head, split)
  // units where their number allows, so that a unit's rows stay in one L2.
  if (units % 8 == 0) {
    const int i = b / 8;
    unit = b % 8 + 8 * (i / tiles);
    t = i % tiles;
  } else if (8 % units == 0) {
    unit = b % 8 % units;
    t = b / 8 * (8 / units) + b % 8 / units;
  } else {
    unit = b % units;
    t = b / units;
  }
  if (t >= tiles || unit >= units) return w;
  t = tiles - 1 - t;   // causal: the long columns come first
  w.head = unit % a.hk;
  w.split = unit / a.hk;
  const int* off = KEYS ? a.seg_k : a.seg_q;
  const int mul = KEYS ? 1 : a.G;
  int lo = 0, hi = a.S;
  while (hi - lo > 1) {
    const int step = (hi - lo + 63) / 64;
    const int s = lo + (int)(threadIdx.x % 64) * step;
    const bool le = s < hi && tile_start(off, s, mul, cols) <= t;
    const int n = max(1, __popcll(__ballot(le)));   // offsets out of order stay in range
    lo += (n - 1) * step;
    hi = min(hi, lo + step);
  }
  w.seg = __builtin_amdgcn_readfirstlane(lo);
  w.tile = t - (int)tile_start(off, w.seg, mul, cols);
  // offsets are clamped to the arrays: bad ones give wrong rows, not bad reads
  auto clamp = [](int x, int l, int h) { return min(max(x, l), h); };
  w.q0 = a.seg_q ? clamp(a.seg_q[w.seg], 0, a.nq) : 0;
  w.lq = (a.seg_q ? clamp(a.seg_q[w.seg + 1], w.q0, a.nq) : a.nq) - w.q0;
  w.k0 = a.seg_k ? clamp(a.seg_k[w.seg], 0, a.nk) : 0;
  w.lk = (a.seg_k ? clamp(a.seg_k[w.seg + 1], w.k0, a.nk) : a.nk) - w.k0;
  w.pre = a.causal && a.prefix ? clamp(a.prefix[w.seg], 0, w.lk) : 0;
  w.any = w.tile >= 0 && (int64_t)w.tile * cols < (int64_t)(KEYS ? w.lk : w.lq) * mul;
  return w;
}

// number of keys that query i of the segment sees (the first ones)
__device__ __forceinline__ int visible(const AttnArgs& a, const Work& w, int i) {
  return a.causal ? min(w.lk, max(w.pre, max(0, i + (w.lk - w.lq) + 1))) : w.lk;
}

// part `split` of [0, n) in multiples of `unit`
__device__ __forceinline__ void split_range(int n, int unit, int splits, int split, int& lo, int& hi) {
  const int per = ((n + splits - 1) / splits + unit - 1) / unit * unit;
  lo = min(n, split * per);
  hi = min(n, lo + per);
}

// Key positions of a tile, one array per coordinate.
template <int ROWS>
struct PosTile {
  float x[ROWS], y[ROWS], z[ROWS];
};

__device__ __forceinline__ f32x4 four(const float* p) { return *reinterpret_cast<const f32x4*>(p); }

// ---------------------------------------------------------------- forward --

template <class T, int DP, int NW, int NS, bool BIAS, bool CAP>
__global__ __launch_bounds__(NW * 64) void attn_fwd_kernel(AttnArgs a, AttnPart part, int tiles) {
  using TL = Tile<T, DP>;
  constexpr int ROWS = 32 * NS, COLS = 32 * NW, TH = NW * 64;
  __shared__ __align__(16) T lk[ROWS * TL::LD];
  __shared__ __align__(16) T lv[ROWS * TL::LD];
  __shared__ __align__(16) PosTile<BIAS ? ROWS : 4> lp;
  const Work w = find_work<false>(a, COLS, tiles, part.splits);
  if (!w.any) return;   // the whole block
  const int lane = threadIdx.x % 64, wv = threadIdx.x / 64, h = lane / 32;
  const int col = w.tile * COLS + wv * 32 + lane % 32;
  const int i = col / a.G, head = w.head * a.G + col % a.G;
  const bool live = i < w.lq;
  const size_t qrow = w.q0 + i;
  typename TL::Frag qf[TL::STEPS];
  TL::load_cols(static_cast<const T*>(a.q) + (live ? qrow * a.qs + (size_t)head * a.D : 0), live, a.D, h, qf);
  float px = 0.f, py = 0.f, pz = 0.f, slope = 0.f;
  if (BIAS && live) {
    px = a.pos_q[3 * qrow], py = a.pos_q[3 * qrow + 1], pz = a.pos_q[3 * qrow + 2];
    slope = a.slope[head] * kLog2e;
  }
  const int vis = live ? visible(a, w, i) : 0;
  // the last column of the block sees the most
  const int iend = min(w.lq, (w.tile * COLS + COLS - 1) / a.G + 1);
  int kb, ke;
  split_range(visible(a, w, iend - 1), ROWS, part.splits, w.split, kb, ke);
  const float c1 = CAP ? a.scale / a.cap : a.scale * kLog2e, c2 = a.cap * kLog2e;

  f32x16 o[TL::DB];
#pragma unroll
  for (int b = 0; b < TL::DB; ++b) o[b] = f32x16{};
  float m = -kInf, l = 0.f;

  Stage<T, DP, ROWS, TH> sk, sv;
  float sp[3] = {0.f, 0.f, 0.f};
  const T* kbase = static_cast<const T*>(a.k) + (size_t)w.k0 * a.ks + (size_t)w.head * a.D;
  const T* vbase = static_cast<const T*>(a.v) + (size_t)w.k0 * a.vs + (size_t)w.head * a.D;
  auto fetch = [&](int j0) {
    sk.load(a.D, [&](int r) { return j0 + r < ke ? kbase + (size_t)(j0 + r) * a.ks : nullptr; });
    sv.load(a.D, [&](int r) { return j0 + r < ke ? vbase + (size_t)(j0 + r) * a.vs : nullptr; });
    if (BIAS && threadIdx.x < ROWS)
#pragma unroll
      for (int c = 0; c < 3; ++c)
        sp[c] = j0 + (int)threadIdx.x < ke ? a.pos_k[3 * (size_t)(w.k0 + j0 + threadIdx.x) + c] : 0.f;
  };
  if (kb < ke) fetch(kb);
  for (int j0 = kb; j0 < ke; j0 += ROWS) {
    __syncthreads();   // the tile before has been read
    sk.store(lk);
    sv.store(lv);
    if (BIAS && threadIdx.x < ROWS) lp.x[threadIdx.x] = sp[0], lp.y[threadIdx.x] = sp[1], lp.z[threadIdx.x] = sp[2];
    __syncthreads();
    if (j0 + ROWS < ke) fetch(j0 + ROWS);

    f32x16 s[NS];
#pragma unroll
    for (int n = 0; n < NS; ++n) s[n] = TL::dot(lk + n * 32 * TL::LD, qf, lane);
    // scores in units of log 2
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        f32x4 kx, ky, kz;
        if constexpr (BIAS) {
          const int j = n * 32 + r4 * 8 + h * 4;
          kx = four(lp.x + j), ky = four(lp.y + j), kz = four(lp.z + j);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = s[n][r4 * 4 + e] * c1;
          if constexpr (CAP) x = c2 * tanh_fast(x);
          if constexpr (BIAS) {
            const float dx = px - kx[e], dy = py - ky[e], dz = pz - kz[e];
            x = fmaf(-slope, __builtin_amdgcn_sqrtf(fmaf(dx, dx, fmaf(dy, dy, dz * dz))), x);
          }
          s[n][r4 * 4 + e] = x;
        }
      }
    if (__any(j0 + ROWS > vis))
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (j0 + n * 32 + acc_row(r, h) >= vis) s[n][r] = -kInf;
    float mx = s[0][0];
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
      for (int r = 0; r < 16; ++r) mx = fmaxf(mx, s[n][r]);
    mx = fmaxf(mx, other_half(mx));
    if (__any(mx > m)) {
      // a new maximum for some column: what was added so far shrinks
      const float mn = fmaxf(m, mx);
      const float f = mn == -kInf ? 1.f : __builtin_amdgcn_exp2f(m - mn);
      m = mn;
      l *= f;
#pragma unroll
      for (int b = 0; b < TL::DB; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[b][r] *= f;
    }
    const float ms = m == -kInf ? 0.f : m;   // nothing seen yet: exp2(-inf) = 0
#pragma unroll
    for (int n = 0; n < NS; ++n) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        s[n][r] = __builtin_amdgcn_exp2f(s[n][r] - ms);
        l += s[n][r];
      }
      TL::outer(lv + n * 32 * TL::LD, s[n], o, lane);
    }
  }
  l += other_half(l);
  if (!live) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const float lse = l == 0.f ? -kInf : (m + __builtin_amdgcn_logf(l)) * kLn2;   // v_log is base 2
  const size_t orow = qrow * a.hq + head;
  if (part.splits == 1) {
    if (h == 0) a.lse[orow] = lse;
    T* dst = static_cast<T*>(a.out) + orow * a.D;
#pragma unroll
    for (int b = 0; b < TL::DB; ++b)
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        const int d = b * 32 + r4 * 8 + h * 4;
        const float x[4] = {o[b][r4 * 4] * inv, o[b][r4 * 4 + 1] * inv, o[b][r4 * 4 + 2] * inv, o[b][r4 * 4 + 3] * inv};
        if (d < a.D) store_f32<T, 4>(dst + d, x);
      }
  } else {
    const size_t prow = (size_t)w.split * a.nq * a.hq + orow;
    if (h == 0) part.lse[prow] = lse;
    float* dst = part.o + prow * a.D;
#pragma unroll
    for (int b = 0; b < TL::DB; ++b)
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        const int d = b * 32 + r4 * 8 + h * 4;
        const float x[4] = {o[b][r4 * 4] * inv, o[b][r4 * 4 + 1] * inv, o[b][r4 * 4 + 2] * inv, o[b][r4 * 4 + 3] * inv};
        if (d < a.D) store_f32<float, 4>(dst + d, x);
      }
  }
}

// ------------------------------------------------- VJP: the scores again --

// From raw products (rows in registers) to P, and for a cap the factor
// 1 - (t / cap)^2; rx.. are the row-to-column differences' source.
template <bool CAP>
__device__ __forceinline__ float score(float u, float c1, float c2, float& th) {
  float x = u * c1;
  if constexpr (CAP) {
    th = tanh_fast(x);
    x = c2 * th;
  }
  return x;
}

// 1 / r with 0 at r = 0, where the distance has no direction
__device__ __forceinline__ float inv_dist(float r2) { return r2 > 0.f ? __builtin_amdgcn_rsqf(r2) : 0.f; }

// ------------------------------------------------- VJP: over query columns --

// DELTA: only delta_i = sum_j P dP into part.delta.  Else q_bar, and the
// position and slope gradients of the query rows into part.row.
template <class T, int DP, int NW, bool BIAS, bool CAP, bool DELTA>
__global__ __launch_bounds__(NW * 64) void attn_query_kernel(AttnArgs a, AttnPart part, int tiles) {
  using TL = Tile<T, DP>;
  constexpr int ROWS = 32, COLS = 32 * NW, TH = NW * 64;
  __shared__ __align__(16) T lk[ROWS * TL::LD];
  __shared__ __align__(16) T lv[ROWS * TL::LD];
  __shared__ __align__(16) PosTile<BIAS ? ROWS : 4> lp;
  const int splits = DELTA ? part.dsplits : part.splits;
  const Work w = find_work<false>(a, COLS, tiles, splits);
  if (!w.any) return;
  const int lane = threadIdx.x % 64, wv = threadIdx.x / 64, h = lane / 32;
  const int col = w.tile * COLS + wv * 32 + lane % 32;
  const int i = col / a.G, head = w.head * a.G + col % a.G;
  const bool live = i < w.lq;
  const size_t qrow = w.q0 + i, orow = qrow * a.hq + head, nrows = (size_t)a.nq * a.hq;
  typename TL::Frag qf[TL::STEPS], gf[TL::STEPS];
  TL::load_cols(static_cast<const T*>(a.q) + (live ? qrow * a.qs + (size_t)head * a.D : 0), live, a.D, h, qf);
  TL::load_cols(static_cast<const T*>(a.g) + (live ? orow * a.D : 0), live, a.D, h, gf);
  float px = 0.f, py = 0.f, pz = 0.f, slope = 0.f;
  if (BIAS && live) {
    px = a.pos_q[3 * qrow], py = a.pos_q[3 * qrow + 1], pz = a.pos_q[3 * qrow + 2];
    slope = a.slope[head] * kLog2e;
  }
  const int vis = live ? visible(a, w, i) : 0;
  // an empty row has lse = -inf; +inf makes its P vanish
  float lse = live ? a.lse[orow] * kLog2e : kInf;
  if (lse == -kInf) lse = kInf;
  float delta = 0.f;
  if (!DELTA && live)
    for (int s = 0; s < part.dsplits; ++s) delta += part.delta[(size_t)s * nrows + orow];
  const int iend = min(w.lq, (w.tile * COLS + COLS - 1) / a.G + 1);
  int kb, ke;
  split_range(visible(a, w, iend - 1), ROWS, splits, w.split, kb, ke);
  const float c1 = CAP ? a.scale / a.cap : a.scale * kLog2e, c2 = a.cap * kLog2e;

  f32x16 dq[TL::DB];
#pragma unroll
  for (int b = 0; b < TL::DB; ++b) dq[b] = f32x16{};
  float gx = 0.f, gy = 0.f, gz = 0.f, gs = 0.f, dsum = 0.f;

  Stage<T, DP, ROWS, TH> sk, sv;
  float sp[3] = {0.f, 0.f, 0.f};
  const T* kbase = static_cast<const T*>(a.k) + (size_t)w.k0 * a.ks + (size_t)w.head * a.D;
  const T* vbase = static_cast<const T*>(a.v) + (size_t)w.k0 * a.vs + (size_t)w.head * a.D;
  auto fetch = [&](int j0) {
    sk.load(a.D, [&](int r) { return j0 + r < ke ? kbase + (size_t)(j0 + r) * a.ks : nullptr; });
    sv.load(a.D, [&](int r) { return j0 + r < ke ? vbase + (size_t)(j0 + r) * a.vs : nullptr; });
    if (BIAS && threadIdx.x < ROWS)
#pragma unroll
      for (int c = 0; c < 3; ++c)
        sp[c] = j0 + (int)threadIdx.x < ke ? a.pos_k[3 * (size_t)(w.k0 + j0 + threadIdx.x) + c] : 0.f;
  };
  if (kb < ke) fetch(kb);
  for (int j0 = kb; j0 < ke; j0 += ROWS) {
    __syncthreads();
    sk.store(lk);
    sv.store(lv);
    if (BIAS && threadIdx.x < ROWS) lp.x[threadIdx.x] = sp[0], lp.y[threadIdx.x] = sp[1], lp.z[threadIdx.x] = sp[2];
    __syncthreads();
    if (j0 + ROWS < ke) fetch(j0 + ROWS);

    f32x16 s = TL::dot(lk, qf, lane);
    const f32x16 dp = TL::dot(lv, gf, lane);
    const bool edge = __any(j0 + ROWS > vis);
#pragma unroll
    for (int r4 = 0; r4 < 4; ++r4) {
      f32x4 kx, ky, kz;
      if constexpr (BIAS) {
        const int j = r4 * 8 + h * 4;
        kx = four(lp.x + j), ky = four(lp.y + j), kz = four(lp.z + j);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = r4 * 4 + e;
        float th = 0.f, x = score<CAP>(s[r], c1, c2, th);
        float dx, dy, dz, dist, inv;
        if constexpr (BIAS) {
          dx = px - kx[e], dy = py - ky[e], dz = pz - kz[e];
          const float r2 = fmaf(dx, dx, fmaf(dy, dy, dz * dz));
          inv = inv_dist(r2);
          dist = r2 * inv;
          x = fmaf(-slope, dist, x);
        }
        if (edge && j0 + acc_row(r, h) >= vis) x = -kInf;
        const float p = __builtin_amdgcn_exp2f(x - lse);
        if constexpr (DELTA) {
          dsum = fmaf(p, dp[r], dsum);
        } else {
          float ds = p * (dp[r] - delta);
          if constexpr (BIAS) {
            gs = fmaf(ds, dist, gs);
            const float f = ds * inv;
            gx = fmaf(f, dx, gx), gy = fmaf(f, dy, gy), gz = fmaf(f, dz, gz);
          }
          if constexpr (CAP) ds *= 1.f - th * th;
          s[r] = ds;
        }
      }
    }
    if constexpr (!DELTA) TL::outer(lk, s, dq, lane);
  }
  if constexpr (DELTA) {
    dsum += other_half(dsum);
    if (live && h == 0) part.delta[(size_t)w.split * nrows + orow] = dsum;
    return;
  }
  if constexpr (BIAS) {
    gx += other_half(gx), gy += other_half(gy), gz += other_half(gz), gs += other_half(gs);
    if (part.row && live && h == 0) {
      const float t = -slope * kLn2;
      const float x[4] = {t * gx, t * gy, t * gz, -gs};
      store_f32<float, 4>(part.row + ((size_t)w.split * nrows + orow) * 4, x);
    }
  }
  if (!live || !a.gq) return;
#pragma unroll
  for (int b = 0; b < TL::DB; ++b)
#pragma unroll
    for (int r4 = 0; r4 < 4; ++r4) {
      const int d = b * 32 + r4 * 8 + h * 4;
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = dq[b][r4 * 4 + e] * a.scale;
      if (d >= a.D) continue;
      if (part.splits == 1)
        store_f32<T, 4>(static_cast<T*>(a.gq) + orow * a.D + d, x);
      else
        store_f32<float, 4>(part.o + ((size_t)w.split * nrows + orow) * a.D + d, x);
    }
}

// --------------------------------------------------- VJP: over key columns --

template <int ROWS>
struct QueryTile {
  float lse[ROWS], delta[ROWS];
  int vis[ROWS];
};
template <int ROWS>
struct QueryPos {
  float x[ROWS], y[ROWS], z[ROWS], slope[ROWS];
};

template <class T, int DP, int NW, bool BIAS, bool CAP>
__global__ __launch_bounds__(NW * 64) void attn_key_kernel(AttnArgs a, AttnPart part, int tiles) {
  using TL = Tile<T, DP>;
  constexpr int ROWS = 32, COLS = 32 * NW, TH = NW * 64;
  __shared__ __align__(16) T lq[ROWS * TL::LD];
  __shared__ __align__(16) T lg[ROWS * TL::LD];
  __shared__ __align__(16) QueryTile<ROWS> lr;
  __shared__ __align__(16) QueryPos<BIAS ? ROWS : 4> lp;
  const Work w = find_work<true>(a, COLS, tiles, part.splits);
  if (!w.any) return;
  const int lane = threadIdx.x % 64, wv = threadIdx.x / 64, h = lane / 32;
  const int j = w.tile * COLS + wv * 32 + lane % 32;
  const bool live = j < w.lk;
  const size_t krow = w.k0 + j, nrows = (size_t)a.nq * a.hq;
  typename TL::Frag kf[TL::STEPS], vf[TL::STEPS];
  TL::load_cols(static_cast<const T*>(a.k) + (live ? krow * a.ks + (size_t)w.head * a.D : 0), live, a.D, h, kf);
  TL::load_cols(static_cast<const T*>(a.v) + (live ? krow * a.vs + (size_t)w.head * a.D : 0), live, a.D, h, vf);
  float px = 0.f, py = 0.f, pz = 0.f;
  if (BIAS && live) px = a.pos_k[3 * krow], py = a.pos_k[3 * krow + 1], pz = a.pos_k[3 * krow + 2];
  // packed query rows [rb, re): those before the first that sees the block's
  // first key are left out
  const int j0 = w.tile * COLS;
  const int i0 = a.causal && j0 >= w.pre ? min(w.lq, max(0, j0 - (w.lk - w.lq))) : 0;
  const int rows = (w.lq - i0) * a.G;
  int rb, re;
  split_range(rows, ROWS, part.splits, w.split, rb, re);
  rb += i0 * a.G, re += i0 * a.G;
  const float c1 = CAP ? a.scale / a.cap : a.scale * kLog2e, c2 = a.cap * kLog2e;

  f32x16 dk[TL::DB], dv[TL::DB];
#pragma unroll
  for (int b = 0; b < TL::DB; ++b) dk[b] = f32x16{}, dv[b] = f32x16{};
  float gx = 0.f, gy = 0.f, gz = 0.f;

  Stage<T, DP, ROWS, TH> sq, sg;
  float s_lse = kInf, s_delta = 0.f, sp[4] = {0.f, 0.f, 0.f, 0.f};
  int s_vis = 0;
  const T* qbase = static_cast<const T*>(a.q) + (size_t)w.q0 * a.qs + (size_t)w.head * a.G * a.D;
  const T* gbase = static_cast<const T*>(a.g) + ((size_t)w.q0 * a.hq + (size_t)w.head * a.G) * a.D;
  auto fetch = [&](int r0) {
    sq.load(a.D, [&](int r) {
      const int c = r0 + r, i = c / a.G;
      return c < re ? qbase + (size_t)i * a.qs + (size_t)(c - i * a.G) * a.D : nullptr;
    });
    sg.load(a.D, [&](int r) {
      const int c = r0 + r, i = c / a.G;
      return c < re ? gbase + ((size_t)i * a.hq + (c - i * a.G)) * a.D : nullptr;
    });
    if (threadIdx.x < ROWS) {
      const int c = r0 + threadIdx.x, i = c / a.G, head = w.head * a.G + (c - i * a.G);
      const bool on = c < re;
      const size_t orow = (size_t)(w.q0 + i) * a.hq + head;
      s_lse = on ? a.lse[orow] * kLog2e : kInf;
      if (s_lse == -kInf) s_lse = kInf;   // an empty row: P = 0
      s_delta = 0.f;
      if (on)
        for (int s = 0; s < part.dsplits; ++s) s_delta += part.delta[(size_t)s * nrows + orow];
      s_vis = on ? visible(a, w, i) : 0;
      if constexpr (BIAS) {
#pragma unroll
        for (int k = 0; k < 3; ++k) sp[k] = on ? a.pos_q[3 * (size_t)(w.q0 + i) + k] : 0.f;
        sp[3] = on ? a.slope[head] * kLog2e : 0.f;
      }
    }
  };
  if (rb < re) fetch(rb);
  for (int r0 = rb; r0 < re; r0 += ROWS) {
    __syncthreads();
    sq.store(lq);
    sg.store(lg);
    if (threadIdx.x < ROWS) {
      lr.lse[threadIdx.x] = s_lse, lr.delta[threadIdx.x] = s_delta, lr.vis[threadIdx.x] = s_vis;
      if constexpr (BIAS)
        lp.x[threadIdx.x] = sp[0], lp.y[threadIdx.x] = sp[1], lp.z[threadIdx.x] = sp[2], lp.slope[threadIdx.x] = sp[3];
    }
    __syncthreads();
    if (r0 + ROWS < re) fetch(r0 + ROWS);

    f32x16 s = TL::dot(lq, kf, lane);
    f32x16 dp = TL::dot(lg, vf, lane);
#pragma unroll
    for (int r4 = 0; r4 < 4; ++r4) {
      const int rr = r4 * 8 + h * 4;
      const f32x4 lse = four(lr.lse + rr), delta = four(lr.delta + rr);
      const i32x4 vis = *reinterpret_cast<const i32x4*>(lr.vis + rr);
      f32x4 qx, qy, qz, sl;
      if constexpr (BIAS) qx = four(lp.x + rr), qy = four(lp.y + rr), qz = four(lp.z + rr), sl = four(lp.slope + rr);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = r4 * 4 + e;
        float th = 0.f, x = score<CAP>(s[r], c1, c2, th);
        float dx, dy, dz, inv;
        if constexpr (BIAS) {
          dx = px - qx[e], dy = py - qy[e], dz = pz - qz[e];
          const float r2 = fmaf(dx, dx, fmaf(dy, dy, dz * dz));
          inv = inv_dist(r2);
          x = fmaf(-sl[e], r2 * inv, x);
        }
        if (j >= vis[e]) x = -kInf;
        const float p = __builtin_amdgcn_exp2f(x - lse[e]);
        float ds = p * (dp[r] - delta[e]);
        if constexpr (BIAS) {
          const float f = ds * inv * sl[e];
          gx = fmaf(f, dx, gx), gy = fmaf(f, dy, gy), gz = fmaf(f, dz, gz);
        }
        if constexpr (CAP) ds *= 1.f - th * th;
        s[r] = p;
        dp[r] = ds;
      }
    }
    TL::outer(lg, s, dv, lane);
    TL::outer(lq, dp, dk, lane);
  }
  const size_t orow = krow * a.hk + w.head, knum = (size_t)a.nk * a.hk;
  if constexpr (BIAS) {
    gx += other_half(gx), gy += other_half(gy), gz += other_half(gz);
    if (part.col && live && h == 0) {
      const float x[4] = {-kLn2 * gx, -kLn2 * gy, -kLn2 * gz, 0.f};
      store_f32<float, 4>(part.col + ((size_t)w.split * knum + orow) * 4, x);
    }
  }
  if (!live) return;
#pragma unroll
  for (int b = 0; b < TL::DB; ++b)
#pragma unroll
    for (int r4 = 0; r4 < 4; ++r4) {
      const int d = b * 32 + r4 * 8 + h * 4;
      if (d >= a.D) continue;
      float x[4], y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = dk[b][r4 * 4 + e] * a.scale, y[e] = dv[b][r4 * 4 + e];
      if (part.splits == 1) {
        if (a.gk) store_f32<T, 4>(static_cast<T*>(a.gk) + orow * a.D + d, x);
        if (a.gv) store_f32<T, 4>(static_cast<T*>(a.gv) + orow * a.D + d, y);
      } else {
        const size_t at = ((size_t)w.split * knum + orow) * a.D + d;
        if (a.gk) store_f32<float, 4>(part.o + at, x);
        if (a.gv) store_f32<float, 4>(part.o2 + at, y);
      }
    }
}

// ---------------------------------------------------------------- launches --

template <class T, int DP, int NW>
void attn_launch_nw(const AttnLaunch& l, const AttnArgs& a, const AttnPart& p, hipStream_t st) {
  constexpr int NS = sizeof(T) == 2 ? 2 : 1;
  const bool keys = l.pass == kAttnKey;
  const int splits = l.pass == kAttnDelta ? p.dsplits : p.splits;
  const int64_t cols = 32 * NW;
  const int tiles = (int)((keys ? (int64_t)a.nk : (int64_t)a.nq * a.G) / cols + a.S);
  const int64_t units = (int64_t)a.hk * splits;
  int64_t blocks;
  if (units % 8 == 0)
    blocks = units * tiles;
  else if (8 % units == 0)
    blocks = 8 * ((tiles + 8 / units - 1) / (8 / units));
  else
    blocks = units * tiles;
  const dim3 grid((unsigned)blocks), block(NW * 64);
  auto go = [&](auto bias, auto cap) {
    constexpr bool B = decltype(bias)::value, C = decltype(cap)::value;
    switch (l.pass) {
      case kAttnFwd: hipLaunchKernelGGL((attn_fwd_kernel<T, DP, NW, NS, B, C>), grid, block, 0, st, a, p, tiles); break;
      case kAttnDelta:
        if constexpr (sizeof(T) == 2 && B)   // fp32 rows take delta from out
          hipLaunchKernelGGL((attn_query_kernel<T, DP, NW, B, C, true>), grid, block, 0, st, a, p, tiles);
        break;
      case kAttnQuery:
        hipLaunchKernelGGL((attn_query_kernel<T, DP, NW, B, C, false>), grid, block, 0, st, a, p, tiles);
        break;
      default: hipLaunchKernelGGL((attn_key_kernel<T, DP, NW, B, C>), grid, block, 0, st, a, p, tiles); break;
    }
  };
  using Yes = std::integral_constant<bool, true>;
  using No = std::integral_constant<bool, false>;
  if (a.slope)
    a.cap > 0.f ? go(Yes{}, Yes{}) : go(Yes{}, No{});
  else
    a.cap > 0.f ? go(No{}, Yes{}) : go(No{}, No{});
}

template <class T, int DP>
void attn_launch(const AttnLaunch& l, const AttnArgs& a, const AttnPart& p, hipStream_t st) {
  l.waves == 1 ? attn_launch_nw<T, DP, 1>(l, a, p, st) : attn_launch_nw<T, DP, 4>(l, a, p, st);
}

}  // namespace fc
