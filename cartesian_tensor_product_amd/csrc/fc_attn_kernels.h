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
// (ds_read_b64_tr_b16).
//
// fp32 rows are split into three bfloat16 parts, x = h + m + l without a
// remainder, and a product of two of them into the six partial products down
// to 2^-16 of the largest (the three left out are below 2^-25).  The fp32
// matrix instruction runs on the vector units: per 32 x 32 x 2 it takes 74
// cycles during which no vector instruction issues, 592 for a depth of 16; six
// bfloat16 ones take 222 and vector work goes on meanwhile.
//
// Bound by the vector units, which form the scores' tanh, distance, exponential
// and parts, and by latency where registers leave one or two waves per SIMD.
// Measured, forward / query pass / key pass:
//   4096 rows, 4 heads of 32, fp32, slopes: 77 / 120 / 150 us (vector units 58 %
//   busy, matrix units 30 %; 30 GFLOP in 328 us with the joins, 92 TFLOP/s; the
//   fp32 matrix product of the library runs at 151);
//   384 molecules of 5 .. 120 atoms, 8 heads of 16, fp32, slopes: 46 / 60 / 77 us
//   (vector units 40 .. 50 % busy);
//   7 packed causal segments of 300 .. 2500 rows, 16 / 4 heads of 128, bfloat16,
//   cap: 86 / 119 / 224 us (matrix units 22 / 24 / 17 % busy; the key pass has one
//   wave per SIMD, whose waits nothing covers);
//   16384 rows, 8 heads of 64, bfloat16, slopes, forward: 1.00 ms, 549 TFLOP/s
//   (vector units 60 % busy, two waves per SIMD).
//
// No atomics: each output has one writer, and the VJP is two passes, which
// repeats the scores (seven products instead of five) but keeps results
// bitwise reproducible.
#pragma once

#include <hip/hip_runtime.h>

#include "fc_attn.h"
#include "fc_common.h"
#include "fc_types.h"

namespace fc {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

inline constexpr float kLog2e = 1.44269504088896340736f;
inline constexpr float kLn2 = 0.69314718055994530942f;
inline constexpr float kInf = __builtin_huge_valf();

// 16 bytes of a row in memory: the unit of every load.  In LDS and in the
// columns' registers there are bfloat16 parts, one or three.
template <class T>
constexpr int kPieceOf = 16 / (int)sizeof(T);
template <class T>
constexpr int kParts = sizeof(T) == 4 ? 3 : 1;

__device__ __forceinline__ f32x16 mma(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
// acc += the small products of the parts of a and b.  They have a sum of
// their own where it can be had (the matrix unit drops low bits of a term far
// below its accumulator, towards minus infinity: a bias in long sums).
__device__ __forceinline__ f32x16 mma_low(const bf16x8 (&a)[3], const bf16x8 (&b)[3], f32x16 c) {
  c = mma(a[1], b[1], c);
  c = mma(a[0], b[2], c);
  c = mma(a[2], b[0], c);
  c = mma(a[0], b[1], c);
  return mma(a[1], b[0], c);
}

// x as bfloat16 parts, each rounded to nearest (one: the only rounding).  Two
// elements at a time: one conversion for both, and a part is its upper half.
template <int NP, int N, class V>
__device__ __forceinline__ void split(const float (&x)[N], V (&p)[NP]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    f32x2 r = {x[i], x[i + 1]};
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const bf16x2 b = __builtin_convertvector(r, bf16x2);
      p[k][i] = b[0], p[k][i + 1] = b[1];
      if (k + 1 < NP) {
        const uint32_t u = __builtin_bit_cast(uint32_t, b);
        r[0] -= __builtin_bit_cast(float, u << 16);
        r[1] -= __builtin_bit_cast(float, u & 0xffff0000u);
      }
    }
  }
}

// A batch of reads from LDS stays before the matrix instructions that use it, so
// that one latency is waited for and not one per instruction (bfloat16 rows: 7
// packed segments of 300 .. 2500 rows, 16 / 4 heads of 128, forward and VJP 423 us
// without, 392 us with; fp32 rows have six instructions per read and gain nothing).
__device__ __forceinline__ void reads_first() { __builtin_amdgcn_sched_barrier(0x476); }

// Row of register r of the 32x32 result, for the wave's half h.
__device__ __forceinline__ constexpr int acc_row(int r, int h) { return (r / 4) * 8 + h * 4 + r % 4; }

// A tile of rows in LDS holds HB neighbouring heads of DP elements (padded
// head dimension) per row.  The row length in LDS is an odd multiple of 16
// bytes, so that 16 rows' chunks at one place spread over all banks; rows of
// 256 bytes get 48 more rather than 16, so that also the four rows of a
// transposing read meet at most in pairs.
template <class T, int DP, int HB>
struct Tile {
  static constexpr int NP = kParts<T>, CH = kPieceOf<T>;
  static constexpr int STEPS = DP / 16;                // products over d
  static constexpr int DB = (DP + 31) / 32;            // 32-wide blocks of d
  static constexpr int W = HB * DP;
  static constexpr int LD = W + (DP < 32 ? 32 - DP : 0) + (W == 128 ? 24 : 8);
  static constexpr int CPR = W / CH;                   // pieces of a row
  static constexpr int PART = 32 * LD;                 // one part of 32 rows
  static constexpr int AHEAD = NP == 1 ? STEPS : 1;    // steps and
  static constexpr int BLOCKS = NP == 1 ? DB : 1;      // blocks read at once
  struct Cols {
    bf16x8 f[STEPS][NP];
  };

  // columns of a wave: lane -> its column's elements 16 s + 8 h ...
  static __device__ __forceinline__ void load_cols(const T* row, bool live, int D, int h, Cols& c) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int d = 16 * s + 8 * h;
      const bool in = live && d < D;
      if constexpr (NP == 1) {
        const bf16x8 z = {};
        c.f[s][0] = in ? *reinterpret_cast<const bf16x8*>(row + d) : z;
      } else {
        const f32x4 z = {};
        const f32x4 lo = in ? *reinterpret_cast<const f32x4*>(row + d) : z;
        const f32x4 hi = in ? *reinterpret_cast<const f32x4*>(row + d + 4) : z;
        const float x[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        split(x, c.f[s]);
      }
    }
  }

  // acc[row][col] = sum_d rows[row][d] cols[col][d] for 32 rows in LDS
  static __device__ __forceinline__ f32x16 dot(const bf16* rows, const Cols& cols, int lane) {
    f32x16 c = {}, low = {};
    const bf16* p = rows + (lane % 32) * LD + (lane / 32) * 8;
#pragma unroll
    for (int s0 = 0; s0 < STEPS; s0 += AHEAD) {
      bf16x8 a[AHEAD][NP];
#pragma unroll
      for (int s = 0; s < AHEAD; ++s)
#pragma unroll
        for (int k = 0; k < NP; ++k) a[s][k] = *reinterpret_cast<const bf16x8*>(p + k * PART + 16 * (s0 + s));
      if constexpr (NP == 1) reads_first();
#pragma unroll
      for (int s = 0; s < AHEAD; ++s) {
        if constexpr (NP == 3) low = mma_low(a[s], cols.f[s0 + s], low);
        c = mma(a[s][0], cols.f[s0 + s][0], c);
      }
    }
    if constexpr (NP == 3) c += low;
    return c;
  }

  // out[d][col] += sum_row rows[row][d] w[row][col] for 32 rows in LDS; the
  // weights are taken as WP parts
  template <int WP>
  static __device__ __forceinline__ void outer(const bf16* rows, const f32x16& w, f32x16 (&out)[DB], int lane) {
    // 16 lanes read four rows x 16 columns and get a column each
    const bf16* p = rows + ((lane / 32) * 4 + (lane % 16) / 4) * LD + ((lane / 16) % 2) * 16 + (lane % 4) * 4;
    typedef __attribute__((address_space(3))) i16x4* lds_ptr;
    auto read = [&](int s, int b, int k) {
      const bf16* pb = p + k * PART + s * 16 * LD + b * 32;
      const bf16x4 lo = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(pb)));
      const bf16x4 hi = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(pb + 8 * LD)));
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = w[8 * s + i];
      bf16x8 wb[WP];
      split(x, wb);
#pragma unroll
      for (int b0 = 0; b0 < DB; b0 += BLOCKS) {
        bf16x8 a[BLOCKS][NP];
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
          for (int k = 0; k < NP; ++k) a[b][k] = read(s, b0 + b, k);
        if constexpr (NP == 1) reads_first();
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) {
          if constexpr (NP == 3) out[b0 + b] = mma_low(a[b], wb, out[b0 + b]);
          if constexpr (WP == 2) out[b0 + b] = mma(a[b][0], wb[1], out[b0 + b]);
          out[b0 + b] = mma(a[b][0], wb[0], out[b0 + b]);
        }
      }
    }
  }
};

// Buffer offsets are 32 bits from a base that moves with the tile; an offset
// of kNowhere lies behind every buffer and reads zeros.
constexpr uint32_t kNowhere = 0x7ffffff0u, kReach = 0x7fffff00u;

// bytes from row `row` to the end of `n` rows of `stride` bytes (the last one
// `last` bytes long), as the reach of a buffer
__device__ __forceinline__ uint32_t reach(int row, int n, int64_t stride, int last) {
  return row < n ? (uint32_t)min((int64_t)kReach, (n - 1 - row) * stride + last) : 0u;
}

// A tile on its way from memory to LDS: loaded into registers while the tile
// before is worked on, then stored.  Loads are buffer loads, without branches:
// what lies behind the segment's last row reads as zero.
template <class T, int DP, int HB, int ROWS, int TH>
struct Stage {
  using TL = Tile<T, DP, HB>;
  static constexpr int N = (ROWS * TL::CPR + TH - 1) / TH;
  static constexpr int STEP = TH / TL::CPR;   // rows from one turn to the next
  static_assert(TH % TL::CPR == 0 && (N == 1 || ROWS * TL::CPR % TH == 0) && ROWS % 32 == 0);
  f32x4 r[N];

  // The thread's place t: tile rows t / CPR + n STEP, and bytes inside a row.
  static __device__ __forceinline__ uint32_t place(int t, int D, int head_stride) {
    const int c = t % TL::CPR, d = c % (DP / TL::CH) * TL::CH;
    return t / TL::CPR < ROWS && d < D ? (uint32_t)(c / (DP / TL::CH) * head_stride + d) * sizeof(T) : kNowhere;
  }
  // row(r): byte offset of tile row r from the buffer's base (below 2^31, so
  // that kNowhere stays out of reach)
  template <class F>
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t buf, int t, uint32_t place, F&& row) {
#pragma unroll
    for (int n = 0; n < N; ++n)
      r[n] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(buf, place + row(t / TL::CPR + n * STEP), 0, 0));
  }
  // off: place and row of each turn
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t buf, const uint32_t (&off)[N]) {
#pragma unroll
    for (int n = 0; n < N; ++n)
      r[n] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(buf, off[n], 0, 0));
  }
  // 32 rows after 32 rows, each with its parts
  __device__ __forceinline__ void store(int t, bf16* lds) const {
    if (ROWS * TL::CPR < TH && t >= ROWS * TL::CPR) return;
    const int col = t % TL::CPR * TL::CH;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int row = t / TL::CPR + n * STEP;
      bf16* p = lds + row / 32 * (TL::NP * TL::PART) + row % 32 * TL::LD + col;
      if constexpr (TL::NP == 1) {
        *reinterpret_cast<f32x4*>(p) = r[n];
      } else {
        const float x[4] = {r[n][0], r[n][1], r[n][2], r[n][3]};
        bf16x4 s[TL::NP];
        split(x, s);
#pragma unroll
        for (int k = 0; k < TL::NP; ++k) *reinterpret_cast<bf16x4*>(p + k * TL::PART) = s[k];
      }
    }
  }
};

// Keeps what depends on x inside its branch (few tiles have an edge).
__device__ __forceinline__ int opaque(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

__device__ __forceinline__ float other_half(float x) { return __shfl_xor(x, 32); }
__device__ __forceinline__ f32x4 four(const float* p) { return *reinterpret_cast<const f32x4*>(p); }

// The capped score cap tanh(u / cap) / log 2 - ref of a raw product, and the
// derivative's factor 1 - tanh^2.  EXACT: tanh within a few 2^-24 of its value
// also near 0.  Else, with w = 1 / (1 + exp(2 u / cap)), it is c2 - ref - 2 c2 w,
// and the factor 4 w (1 - w): a third of the work, for an error of a few 2^-24
// cap, which is taken where bfloat16 weights are rounded to 2^-9 anyway
// (kWeightParts of 1).
template <bool EXACT>
struct Cap {
  float c1, c2;   // scale / cap (else: times 2 / log 2), cap / log 2
  __device__ __forceinline__ Cap(float scale, float cap)
      : c1(scale / cap * (!EXACT ? 2.f * kLog2e : 1.f)), c2(cap * kLog2e) {}
  __device__ __forceinline__ float score(float u, float ref, float& t) const {
    if constexpr (!EXACT) {
      t = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(u * c1));
      return fmaf(-2.f * c2, t, c2 - ref);
    } else {
      const float x = u * c1, z = x * x;   // Taylor series; |x| < 0.4 leaves z^7 below 2^-24
      float p = fmaf(z, 21844.f / 6081075.f, -1382.f / 155925.f);
      p = fmaf(z, p, 62.f / 2835.f);
      p = fmaf(z, p, -17.f / 315.f);
      p = fmaf(z, p, 2.f / 15.f);
      p = fmaf(z, p, -1.f / 3.f);
      const float far = fmaf(-2.f, __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(x * (2.f * kLog2e))), 1.f);
      t = z < 0.16f ? fmaf(x * z, p, x) : far;
      return fmaf(c2, t, -ref);
    }
  }
  // ds (1 - tanh^2), without kRest
  static __device__ __forceinline__ float slope(float ds, float t) {
    if constexpr (!EXACT) return ds * fmaf(-t, t, t);
    return fmaf(-t * t, ds, ds);
  }
  static constexpr float kRest = !EXACT ? 4.f : 1.f;
};

// 1 / r of a squared distance.  Squares carry 1e-35, so that at r = 0 this is
// a large finite value, which meets differences that are 0 there.
__device__ __forceinline__ float inv_dist(float r2) { return __builtin_amdgcn_rsqf(r2); }
// r from it; fp32 rows get a Newton step, since slope r may be tens
template <class T>
__device__ __forceinline__ float dist_of(float r2, float inv) {
  const float r = r2 * inv;
  return sizeof(T) == 2 ? r : fmaf(0.5f * inv, fmaf(-r, r, r2), r);
}

// (a + b) log 2, rounded once: the products' and the sum's rests are kept, since
// an error of lse scales a whole row's probabilities in the VJP
__device__ __forceinline__ float ln_of(float a, float b) {
  constexpr float kLn2Rest = -1.90465429995776804525e-9f;   // log 2 - kLn2
  const float s = a + b, rest = fabsf(a) > fabsf(b) ? (a - s) + b : (b - s) + a;
  const float p = s * kLn2;
  return p + (fmaf(s, kLn2, -p) + fmaf(s, kLn2Rest, rest * kLn2));
}

// lse for the VJP: probabilities are exp2(score - ref) factor with a whole
// number ref, so that the rest of lse / log 2 is not rounded with it.  A row
// that sees no key (lse = -inf) gets ref = inf: its probabilities vanish.
struct Norm {
  float ref, factor;
  __device__ __forceinline__ explicit Norm(float lse) {
    constexpr float kLog2eRest = 1.92596299112661746887e-8f;   // 1 / log 2 - kLog2e
    const float x = lse * kLog2e, rest = fmaf(lse, kLog2e, -x) + lse * kLog2eRest;
    const bool some = fabsf(lse) < kInf;
    ref = some ? rintf(x) : kInf;
    factor = some ? __builtin_amdgcn_exp2f((ref - x) - rest) : 1.f;
  }
};

// Differences and distances from a column's point to four rows' points.
struct Points {
  f32x4 dx, dy, dz;
  __device__ __forceinline__ Points(float px, float py, float pz, const float* x, const float* y, const float* z)
      : dx(px - four(x)), dy(py - four(y)), dz(pz - four(z)) {}
  __device__ __forceinline__ float square(int e) const { return fmaf(dx[e], dx[e], fmaf(dy[e], dy[e], fmaf(dz[e], dz[e], 1e-35f))); }
  // g += f (p - row)
  __device__ __forceinline__ void add(int e, float f, float (&g)[3]) const {
    g[0] = fmaf(f, dx[e], g[0]), g[1] = fmaf(f, dy[e], g[1]), g[2] = fmaf(f, dz[e], g[2]);
  }
};

// ------------------------------------------------- which work a block has --

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

struct Work {
  int tile, head, split;   // column tile in its segment, first key head
  int q0, lq, k0, lk, pre;
  bool any;
};

// Tiles of `cols` columns: segment s starts at tile off[s] mul / cols + s,
// which leaves every segment room for its last, partial tile without a scan
// over the segments before it (at most one tile per segment stays empty).
__device__ __forceinline__ int64_t tile_start(int off, int s, int mul, int cols) {
  return (int64_t)off * mul / cols + s;
}

// The column axis is queries (mul = G) or keys (mul = 1).  All lanes of a
// wave search together.
template <bool KEYS>
__device__ __forceinline__ Work find_work(const AttnArgs& a, int cols, int hb, int tiles, int splits) {
  Work w{};
  const int heads = a.hk / hb, units = heads * splits;
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
  w.head = unit % heads * hb;
  w.split = unit / heads;
  auto clamp = [](int x, int l, int h) { return min(max(x, l), h); };
  const int* off = KEYS ? a.seg_k : a.seg_q;
  const int n = KEYS ? a.nk : a.nq, mul = KEYS ? 1 : a.G, lane = threadIdx.x % 64;
  const int* other = KEYS ? a.seg_q : a.seg_k;
  const int no = KEYS ? a.nq : a.nk;
  int seg = 0, c0 = 0, c1 = n;
  // Of a causal segment the columns with long walks (late queries, early keys)
  // come first.  Where not all blocks run at once, so do the segments with long
  // walks, of up to 16: a long block that starts last would be waited for (7
  // segments of 300 .. 2500 rows, 16 / 4 heads of 128, forward and VJP: 447 us in
  // the segments' order, 408 us).  Sorting them costs half a microsecond.
  if (off && a.S > 1 && a.S <= 16 && tiles * units > 256) {
    const int s = min(lane, a.S - 1);
    const int o0 = clamp(off[s], 0, n), o1 = clamp(off[s + 1], o0, n);
    const int mine = lane < a.S ? (int)(((int64_t)(o1 - o0) * mul + cols - 1) / cols) : 0;
    int walk = o1 - o0;
    if (other != off) {
      const int p0 = other ? clamp(other[s], 0, no) : 0;
      walk = other ? clamp(other[s + 1], p0, no) - p0 : no;
    }
    int start = 0;
    for (int k = 0; k < a.S; ++k) {
      const int wk = __builtin_amdgcn_readlane(walk, k), tk = __builtin_amdgcn_readlane(mine, k);
      start += wk > walk || (wk == walk && k < lane) ? tk : 0;
    }
    const unsigned long long here = __ballot(t >= start && t - start < mine);
    seg = uniform(here == 0 ? 0 : __builtin_ctzll(here));
    w.tile = here == 0 ? -1 : __builtin_amdgcn_readlane(KEYS ? t - start : mine - 1 - (t - start), seg);
    c0 = __builtin_amdgcn_readlane(o0, seg);
    c1 = __builtin_amdgcn_readlane(o1, seg);
  } else if (off) {
    if (!KEYS) t = tiles - 1 - t;
    int lo = 0, hi = a.S;
    while (hi - lo > 63) {   // 64 candidates per step
      const int step = (hi - lo + 63) / 64, s = lo + lane * step;
      const bool le = s < hi && tile_start(off[min(s, hi)], s, mul, cols) <= t;
      lo += (max(1, __popcll(__ballot(le))) - 1) * step;
      hi = min(hi, lo + step);
    }
    const int s = min(lo + lane, hi), o = off[s];
    const bool le = lo + lane < hi && tile_start(o, s, mul, cols) <= t;
    const int at = max(1, __popcll(__ballot(le))) - 1;   // offsets out of order stay in range
    seg = __builtin_amdgcn_readfirstlane(lo + at);
    // offsets are clamped to the arrays: bad ones give wrong rows, not bad reads
    const int o0 = __builtin_amdgcn_readlane(o, at), o1 = __builtin_amdgcn_readlane(o, at + 1);
    w.tile = t - (int)tile_start(o0, seg, mul, cols);
    c0 = clamp(o0, 0, n);
    c1 = clamp(o1, c0, n);
  } else {
    w.tile = KEYS ? t : tiles - 1 - t;
  }
  int r0 = c0, r1 = c1;
  if (other != off) {
    r0 = other ? clamp(other[seg], 0, no) : 0;
    r1 = other ? clamp(other[seg + 1], r0, no) : no;
  } else if (!off) {
    r1 = no;
  }
  w.q0 = uniform(KEYS ? r0 : c0), w.lq = uniform(KEYS ? r1 - r0 : c1 - c0);
  w.k0 = uniform(KEYS ? c0 : r0), w.lk = uniform(KEYS ? c1 - c0 : r1 - r0);
  w.pre = uniform(a.causal && a.prefix ? clamp(a.prefix[seg], 0, w.lk) : 0);
  w.tile = uniform(w.tile);
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

// How the waves of a block share its work.
//  kOne: one wave, 32 columns.  kCols: four waves with 32 columns each, every
//  row tile loaded once for all.  kRows: four waves with the same 32 columns,
//  each with its own row tiles (every fourth), joined through LDS at the end.
template <int MODE>
struct Waves {
  static constexpr int NW = MODE == kOne ? 1 : 4;
  static constexpr int TH = NW * 64;
  static constexpr int COLS = MODE == kCols ? 128 : 32;
  static constexpr int REGIONS = MODE == kRows ? 4 : 1;       // row tiles in LDS
  static constexpr int STAGE = MODE == kCols ? 256 : 64;      // threads that fill one
  static constexpr int STRIDE = MODE == kRows ? 4 : 1;        // tiles from one to the next of a wave
  static __device__ __forceinline__ int stage_thread() { return MODE == kCols ? threadIdx.x : threadIdx.x % 64; }
  static __device__ __forceinline__ int region() { return MODE == kRows ? uniform(threadIdx.x / 64) : 0; }
  // between the writes and the reads of a tile
  static __device__ __forceinline__ void sync() {
    if constexpr (MODE == kCols)
      __syncthreads();
    else   // a wave's LDS accesses are served in order; this holds the compiler
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
};

// Parts of the weights (P, dS) in the second products of bfloat16 rows.  One is
// a rounding of 2^-9 at most to each weight, as large as the output's own.  Two
// bring it down to 2^-17 for one matrix instruction and a split more, which costs
// nothing where a call is bound by latency or its loads (kOne, kRows: 16 rows
// over 16 .. 8192 keys 32.2 us with one part, 33.2 us with two), but 15 to 25 %
// where the vector units are full (kCols: 16384 rows, 8 heads of 64 with slopes
// 1.01 ms and 1.27 ms).  Wide heads of the key pass run as kRows under full
// load, too.
template <class T, int DP, int MODE, bool KEY = false>
constexpr int kWeightParts = sizeof(T) == 4 ? 3 : MODE == kCols || (KEY && DP > 64 && MODE == kRows) ? 1 : 2;

// ------------------------------------------------- results of a wave's columns --

// out(hb, d, x): four elements from d of head hb, for the lane's column
template <int HB, int DB, class F>
__device__ __forceinline__ void each_piece(const f32x16 (&o)[HB][DB], int h, int D, F&& out) {
#pragma unroll
  for (int hb = 0; hb < HB; ++hb)
#pragma unroll
    for (int b = 0; b < DB; ++b)
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        const int d = b * 32 + r4 * 8 + h * 4;
        const float x[4] = {o[hb][b][r4 * 4], o[hb][b][r4 * 4 + 1], o[hb][b][r4 * 4 + 2], o[hb][b][r4 * 4 + 3]};
        if (d < D) out(hb, d, x);
      }
}

// kRows: adds the four waves' results, in wave order.  slices: LDS of the row
// tiles, free by now, `slice` floats per wave.  out(col, hb, d, x) is called
// once per piece, neighbouring threads with neighbouring d.
template <int HB, int DB, class F>
__device__ __forceinline__ void join_waves(float* slices, int slice, const f32x16 (&o)[HB][DB], int D, F&& out) {
  const int lane = threadIdx.x % 64, h = lane / 32, W = HB * D + 4;
  float* mine = slices + threadIdx.x / 64 * slice + lane % 32 * W;
  __syncthreads();
  each_piece(o, h, D, [&](int hb, int d, const float* x) { store_f32<float, 4>(mine + hb * D + d, x); });
  __syncthreads();
  const int per = HB * D / 4;
  for (int e = threadIdx.x; e < 32 * per; e += 256) {
    const int col = e / per, c = (e - col * per) * 4;
    float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      float y[4];
      load_f32<float, 4>(slices + w * slice + col * W + c, y);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] += y[i];
    }
    out(col, c / D, c % D, x);
  }
}

// sum over the four waves of a value per (n, column), in wave order; buf
// holds 4 x N x 32 floats
template <int N>
__device__ __forceinline__ void join_values(float* buf, float (&v)[N]) {
  const int lane = threadIdx.x % 64, w = threadIdx.x / 64;
  __syncthreads();
  if (lane < 32)
#pragma unroll
    for (int i = 0; i < N; ++i) buf[(w * N + i) * 32 + lane] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) t += buf[(k * N + i) * 32 + lane % 32];
    v[i] = t;
  }
}

// Waves per SIMD that a kernel's registers allow: columns and accumulators of
// all heads, `live` 32x32 results at a time, the tile on its way, and what
// goes into addresses, scalars and reads ahead from LDS, out of 512; and that
// the row tiles of their blocks allow, out of 160 KB of LDS.
template <class T, int DP, int HB, int MODE, bool BIAS>
constexpr int waves_per_simd(int frags, int accs, int live, int rows) {
  using TL = Tile<T, DP, HB>;
  const int regs = frags * HB * TL::STEPS * TL::NP * 4 + accs * HB * TL::DB * 16 + live * 16 +
                   2 * 4 * ((rows * TL::CPR + Waves<MODE>::STAGE - 1) / Waves<MODE>::STAGE) + (BIAS ? 100 : 60) +
                   (accs == 2 && TL::NP == 3 ? 40 : 0);
  constexpr int lds = Waves<MODE>::REGIONS * (2 * TL::LD * TL::NP * 2 + (BIAS ? 32 : 16));   // of a tile row
  const int room = (163840 / (lds * rows) * Waves<MODE>::NW + 3) / 4;
  const int waves = regs <= 168 ? 3 : regs <= 256 ? 2 : 1;
  return waves < room ? waves : room > 0 ? room : 1;
}

// ---------------------------------------------------------------- forward --

// The softmax in one pass, in units of log 2.  Scores are formed relative to
// a reference m per column, which follows the running maximum: it is raised
// (and what was added so far is scaled down) at the first tile and when a
// score exceeds it by 2^kSlack, so most tiles need neither a subtraction nor a
// scaling.  The keys a column sees are the first ones, so a column that sees
// none in a wave's first tile sees none at all there.
constexpr float kSlack = 8.f;

template <class T, int HB, int MODE>
constexpr int fwd_rows() {
  return sizeof(T) == 2 && HB == 1 && MODE == kCols ? 64 : 32;
}

template <class T, int DP, int HB, int MODE, bool BIAS, bool CAP>
__global__ __launch_bounds__(Waves<MODE>::TH, (waves_per_simd<T, DP, HB, MODE, BIAS>(1, 1, fwd_rows<T, HB, MODE>() / 32 * (1 + BIAS), fwd_rows<T, HB, MODE>())))
void attn_fwd_kernel(AttnArgs a, AttnPart part, int tiles) {
  using TL = Tile<T, DP, HB>;
  using WV = Waves<MODE>;
  constexpr int WP = kWeightParts<T, DP, MODE>;
  constexpr int ROWS = fwd_rows<T, HB, MODE>(), NS = ROWS / 32;
  constexpr int AREA = ROWS * TL::LD * TL::NP;   // LDS of one row tile
  __shared__ __align__(16) bf16 lds[WV::REGIONS * 2 * AREA];
  __shared__ __align__(16) float lpos[BIAS ? WV::REGIONS * 3 * ROWS : 4];
  const Work w = find_work<false>(a, WV::COLS, HB, tiles, part.splits);
  if (!w.any) return;   // the whole block
  const int lane = threadIdx.x % 64, wv = uniform(threadIdx.x / 64), h = lane / 32, st = WV::stage_thread();
  const int col = w.tile * WV::COLS + (MODE == kCols ? wv * 32 : 0) + lane % 32;
  const int i = col / a.G, head = w.head * a.G + col % a.G;   // + hb G for the other heads
  const bool live = i < w.lq;
  const size_t qrow = w.q0 + i;
  bf16 *lk = lds + WV::region() * 2 * AREA, *lv = lk + AREA;
  float* lp = lpos + (BIAS ? WV::region() * 3 * ROWS : 0);

  const int vis = live ? visible(a, w, i) : 0;
  // the last column of the block sees the most
  const int iend = min(w.lq, (w.tile * WV::COLS + WV::COLS - 1) / a.G + 1);
  int kb, ke;
  split_range(visible(a, w, iend - 1), ROWS, part.splits, w.split, kb, ke);
  if (MODE == kRows) kb += wv * ROWS;

  Stage<T, DP, HB, ROWS, WV::STAGE> sk, sv;
  const uint32_t place = sk.place(st, a.D, a.D);
  float sp[3];
  const T* kbase = static_cast<const T*>(a.k) + (size_t)w.k0 * a.ks + (size_t)w.head * a.D;
  const T* vbase = static_cast<const T*>(a.v) + (size_t)w.k0 * a.vs + (size_t)w.head * a.D;
  const uint32_t kst = (uint32_t)a.ks * sizeof(T), vst = (uint32_t)a.vs * sizeof(T);
  const int row_bytes = HB * a.D * (int)sizeof(T);
  auto fetch = [&](int j0) {
    sk.load(make_rsrc(kbase + (size_t)j0 * a.ks, reach(j0, w.lk, kst, row_bytes)), st, place,
            [&](int r) { return r * kst; });
    sv.load(make_rsrc(vbase + (size_t)j0 * a.vs, reach(j0, w.lk, vst, row_bytes)), st, place,
            [&](int r) { return r * vst; });
    if constexpr (BIAS) {
      const auto buf = make_rsrc(a.pos_k + 3 * (size_t)(w.k0 + j0), reach(j0, w.lk, 12, 12));
#pragma unroll
      for (int c = 0; c < 3; ++c)
        sp[c] = buf_load(buf, st < ROWS ? st * 12 + c * 4 : kNowhere, 0);
    }
  };
  if (kb < ke) fetch(kb);

  typename TL::Cols qf[HB];
  float slope[HB], m[HB], l[HB];
  f32x16 o[HB][TL::DB];
#pragma unroll
  for (int hb = 0; hb < HB; ++hb) {
    const int hq = head + hb * a.G;
    TL::load_cols(static_cast<const T*>(a.q) + (live ? qrow * a.qs + (size_t)hq * a.D : 0), live, a.D, h, qf[hb]);
    slope[hb] = BIAS && live ? a.slope[hq] * kLog2e : 0.f;
    m[hb] = l[hb] = 0.f;
#pragma unroll
    for (int b = 0; b < TL::DB; ++b) o[hb][b] = f32x16{};
  }
  float px = 0.f, py = 0.f, pz = 0.f;
  if (BIAS && live) px = a.pos_q[3 * qrow], py = a.pos_q[3 * qrow + 1], pz = a.pos_q[3 * qrow + 2];
  const float c1 = a.scale * kLog2e;
  const Cap<(WP > 1)> cap(a.scale, a.cap);

  bool first = true;
  auto tile = [&](bool edge, int j0) {
    f32x16 dist[NS];
    if constexpr (BIAS)
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) {
          const float* p = lp + n * 32 + r4 * 8 + h * 4;
          const Points pt(px, py, pz, p, p + ROWS, p + 2 * ROWS);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float r2 = pt.square(e);
            if constexpr (sizeof(T) == 2)
              dist[n][r4 * 4 + e] = __builtin_amdgcn_sqrtf(r2);
            else
              dist[n][r4 * 4 + e] = dist_of<T>(r2, inv_dist(r2));
          }
        }
    f32x16 s[HB][NS];
    float mx[HB];
#pragma unroll
    for (int hb = 0; hb < HB; ++hb) {
#pragma unroll
      for (int n = 0; n < NS; ++n) s[hb][n] = TL::dot(lk + n * TL::NP * TL::PART + hb * DP, qf[hb], lane);
      mx[hb] = -kInf;
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          float x, t;
          if constexpr (CAP)
            x = cap.score(s[hb][n][r], m[hb], t);
          else
            x = fmaf(s[hb][n][r], c1, -m[hb]);
          if constexpr (BIAS) x = fmaf(-slope[hb], dist[n][r], x);
          s[hb][n][r] = x;
        }
    }
    if (edge) {
      const int last = opaque(vis) - j0;
#pragma unroll
      for (int hb = 0; hb < HB; ++hb)
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (n * 32 + acc_row(r, h) >= last) s[hb][n][r] = -kInf;
    }
    bool raise = first;
#pragma unroll
    for (int hb = 0; hb < HB; ++hb) {
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int r = 0; r < 16; ++r) mx[hb] = fmaxf(mx[hb], s[hb][n][r]);
      mx[hb] = fmaxf(mx[hb], other_half(mx[hb]));
      raise |= mx[hb] > kSlack;
    }
    if (__any(raise)) {
#pragma unroll
      for (int hb = 0; hb < HB; ++hb) {
        // whole numbers, so that m has no rest (c2 - m does not round)
        const float up = mx[hb] == -kInf ? 0.f : rintf(first ? mx[hb] : fmaxf(mx[hb], 0.f));
        const float f = __builtin_amdgcn_exp2f(-up);
        m[hb] += up;
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
          for (int r = 0; r < 16; ++r) s[hb][n][r] -= up;
        if (!first) {   // the first tile's factor may be infinite, and meets zeros
          l[hb] *= f;
#pragma unroll
          for (int b = 0; b < TL::DB; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) o[hb][b][r] *= f;
        }
      }
    }
#pragma unroll
    for (int hb = 0; hb < HB; ++hb)
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        float sum = 0.f;   // tile by tile, so that a long row's sum rounds less often
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          s[hb][n][r] = __builtin_amdgcn_exp2f(s[hb][n][r]);
          sum += s[hb][n][r];
        }
        l[hb] += sum;
        TL::template outer<WP>(lv + n * TL::NP * TL::PART + hb * DP, s[hb][n], o[hb], lane);
      }
  };
  for (int j0 = kb; j0 < ke; j0 += ROWS * WV::STRIDE) {
    WV::sync();   // the tile before has been read
    sk.store(st, lk);
    sv.store(st, lv);
    if (BIAS && st < ROWS) lp[st] = sp[0], lp[ROWS + st] = sp[1], lp[2 * ROWS + st] = sp[2];
    WV::sync();
    if (j0 + ROWS * WV::STRIDE < ke) fetch(j0 + ROWS * WV::STRIDE);

    tile(__any(j0 + ROWS > vis), j0);
    first = false;
  }

  float scale[HB], lse[HB];
#pragma unroll
  for (int hb = 0; hb < HB; ++hb) {
    l[hb] += other_half(l[hb]);
    float top = m[hb], f = 1.f, sum = l[hb];
    if constexpr (MODE == kRows) {   // the other waves' references and sums
      float* buf = reinterpret_cast<float*>(lds);
      __syncthreads();
      if (h == 0) buf[wv * 64 + lane] = sum == 0.f ? -kInf : top, buf[wv * 64 + 32 + lane] = sum;
      __syncthreads();
      top = -kInf;
#pragma unroll
      for (int k = 0; k < 4; ++k) top = fmaxf(top, buf[k * 64 + lane % 32]);
      const float ref = top == -kInf ? 0.f : top;
      f = sum == 0.f ? 0.f : __builtin_amdgcn_exp2f(m[hb] - ref);
      sum = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) sum = fmaf(buf[k * 64 + 32 + lane % 32], __builtin_amdgcn_exp2f(buf[k * 64 + lane % 32] - ref), sum);
    }
    scale[hb] = sum == 0.f ? 0.f : f / sum;
    lse[hb] = sum == 0.f ? -kInf : ln_of(top, __builtin_amdgcn_logf(sum));   // v_log is base 2
#pragma unroll
    for (int b = 0; b < TL::DB; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[hb][b][r] *= scale[hb];
  }
  const size_t rows = (size_t)a.nq * a.hq, row0 = part.splits == 1 ? 0 : w.split * rows;
  if (live && h == 0 && (MODE != kRows || wv == 0))
#pragma unroll
    for (int hb = 0; hb < HB; ++hb)
      (part.splits == 1 ? a.lse : part.lse)[row0 + qrow * a.hq + head + hb * a.G] = lse[hb];
  auto put = [&](size_t row, int d, const float* x) {
    if (part.splits == 1)
      store_f32<T, 4>(static_cast<T*>(a.out) + row * a.D + d, x);
    else
      store_f32<float, 4>(part.o + (row0 + row) * a.D + d, x);
  };
  if constexpr (MODE == kRows) {
    join_waves(reinterpret_cast<float*>(lds), AREA, o, a.D,
               [&](int c, int hb, int d, const float* x) {
                 const int cc = w.tile * 32 + c, ii = cc / a.G;
                 if (ii < w.lq) put((w.q0 + (size_t)ii) * a.hq + (w.head + hb) * a.G + cc % a.G, d, x);
               });
  } else {
    each_piece(o, h, a.D, [&](int hb, int d, const float* x) {
      if (live) put(qrow * a.hq + head + hb * a.G, d, x);
    });
  }
}

// ------------------------------------------------- VJP: over query columns --

// DELTA: only delta_i = sum_j P dP into part.delta.  Else q_bar, and the
// position and slope gradients of the query rows into part.row; delta comes
// from the delta pass, or is <g, out>, formed here and left for the key pass.
// A row that sees no more than one tile takes it as the mean of dP there: with
// few keys dP - delta is small beside both, and <g, out> has out's rounding.
// (So a row of one key has dS = 0, not a rest.)
template <class T, int DP, int MODE, bool BIAS, bool CAP, bool DELTA>
__global__ __launch_bounds__(Waves<MODE>::TH, (waves_per_simd<T, DP, 1, MODE, BIAS>(2, !DELTA, 2 + BIAS, 32)))
void attn_query_kernel(AttnArgs a, AttnPart part, int tiles) {
  using TL = Tile<T, DP, 1>;
  using WV = Waves<MODE>;
  constexpr int WP = kWeightParts<T, DP, MODE>;
  constexpr int ROWS = 32;
  constexpr int AREA = ROWS * TL::LD * TL::NP;   // LDS of one row tile
  __shared__ __align__(16) bf16 lds[WV::REGIONS * 2 * AREA];
  __shared__ __align__(16) float lpos[BIAS ? WV::REGIONS * 3 * ROWS : 4];
  const int splits = DELTA ? part.dsplits : part.splits;
  const Work w = find_work<false>(a, WV::COLS, 1, tiles, splits);
  if (!w.any) return;
  const int lane = threadIdx.x % 64, wv = uniform(threadIdx.x / 64), h = lane / 32, st = WV::stage_thread();
  const int col = w.tile * WV::COLS + (MODE == kCols ? wv * 32 : 0) + lane % 32;
  const int i = col / a.G, head = w.head * a.G + col % a.G;
  const bool live = i < w.lq, lead = live && h == 0 && (MODE != kRows || wv == 0);
  const size_t qrow = w.q0 + i, nrows = (size_t)a.nq * a.hq;
  bf16 *lk = lds + WV::region() * 2 * AREA, *lv = lk + AREA;
  float* lp = lpos + (BIAS ? WV::region() * 3 * ROWS : 0);

  const int vis = live ? visible(a, w, i) : 0;
  const int iend = min(w.lq, (w.tile * WV::COLS + WV::COLS - 1) / a.G + 1);
  int kb, ke;
  split_range(visible(a, w, iend - 1), ROWS, splits, w.split, kb, ke);
  if (MODE == kRows) kb += wv * ROWS;

  Stage<T, DP, 1, ROWS, WV::STAGE> sk, sv;
  const uint32_t place = sk.place(st, a.D, a.D);
  float sp[3];
  const T* kbase = static_cast<const T*>(a.k) + (size_t)w.k0 * a.ks + (size_t)w.head * a.D;
  const T* vbase = static_cast<const T*>(a.v) + (size_t)w.k0 * a.vs + (size_t)w.head * a.D;
  const uint32_t kst = (uint32_t)a.ks * sizeof(T), vst = (uint32_t)a.vs * sizeof(T);
  const int row_bytes = a.D * (int)sizeof(T);
  auto fetch = [&](int j0) {
    sk.load(make_rsrc(kbase + (size_t)j0 * a.ks, reach(j0, w.lk, kst, row_bytes)), st, place,
            [&](int r) { return r * kst; });
    sv.load(make_rsrc(vbase + (size_t)j0 * a.vs, reach(j0, w.lk, vst, row_bytes)), st, place,
            [&](int r) { return r * vst; });
    if constexpr (BIAS) {
      const auto buf = make_rsrc(a.pos_k + 3 * (size_t)(w.k0 + j0), reach(j0, w.lk, 12, 12));
#pragma unroll
      for (int c = 0; c < 3; ++c)
        sp[c] = buf_load(buf, st < ROWS ? st * 12 + c * 4 : kNowhere, 0);
    }
  };
  if (kb < ke) fetch(kb);

  typename TL::Cols qf, gf;
  f32x16 dq[1][TL::DB];
  const size_t orow = qrow * a.hq + head;
  TL::load_cols(static_cast<const T*>(a.q) + (live ? qrow * a.qs + (size_t)head * a.D : 0), live, a.D, h, qf);
  TL::load_cols(static_cast<const T*>(a.g) + (live ? orow * a.D : 0), live, a.D, h, gf);
  const float slope = BIAS && live ? a.slope[head] * kLog2e : 0.f;
  const Norm norm(live ? a.lse[orow] : -kInf);   // the factor is the column's own: at the end
  // delta of a column that sees at most one tile is formed there (below); only
  // split 0 (wave 0) meets that tile, and writes part.delta after it
  const bool brief = vis <= ROWS;
  float delta = 0.f;
  if constexpr (!DELTA) {
    if (part.exact) {
      if (!brief)
        for (int s = 0; s < part.dsplits; ++s) delta += part.delta[s * nrows + orow];
    } else {
      // the lane's elements of both rows, as load_cols takes them
      for (int d = 8 * h; !brief && d < a.D; d += 16) {
        float x[8], y[8];
        load_f32<T, 8>(static_cast<const T*>(a.out) + orow * a.D + d, x);
        load_f32<T, 8>(static_cast<const T*>(a.g) + orow * a.D + d, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) delta = fmaf(x[e], y[e], delta);
      }
      delta += other_half(delta);
      if (lead && !brief && w.split == 0) part.delta[orow] = delta;
    }
  }
#pragma unroll
  for (int b = 0; b < TL::DB; ++b) dq[0][b] = f32x16{};
  float px = 0.f, py = 0.f, pz = 0.f;
  if (BIAS && live) px = a.pos_q[3 * qrow], py = a.pos_q[3 * qrow + 1], pz = a.pos_q[3 * qrow + 2];
  const float c1 = a.scale * kLog2e;
  const Cap<(WP > 1)> cap(a.scale, a.cap);
  float v[4] = {0.f, 0.f, 0.f, 0.f}, dsum[1] = {0.f};   // position and slope gradients; delta

  auto tile = [&](bool edge, int j0) {
    float gp[3] = {0.f, 0.f, 0.f}, gs = 0.f, gd = 0.f;   // of this tile: long sums round less often
    f32x16 s = TL::dot(lk, qf, lane);
    const f32x16 dp = TL::dot(lv, gf, lane);
    if (edge && !CAP) {
      const int last = opaque(vis) - j0;
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if (acc_row(r, h) >= last) s[r] = -kInf;
    }
    // weight of register r, element e of the points pt, relative to 2^-ref;
    // its tanh, distance and inverse distance
    auto weight = [&](int r, int e, const Points& pt, float& th, float& d, float& inv) {
      float x;
      if constexpr (CAP) {
        x = cap.score(s[r], norm.ref, th);
        if ((BIAS || DELTA) && edge && j0 + acc_row(r, h) >= vis) x = -kInf;
      } else {
        x = fmaf(s[r], c1, -norm.ref);
      }
      if constexpr (BIAS) {
        inv = inv_dist(pt.square(e));
        d = dist_of<T>(pt.square(e), inv);
        x = fmaf(-slope, d, x);
      }
      return __builtin_amdgcn_exp2f(x);
    };
    auto points = [&](int r4) {
      const float* p = lp + (BIAS ? r4 * 8 + h * 4 : 0);
      return Points(px, py, pz, p, BIAS ? p + ROWS : p, BIAS ? p + 2 * ROWS : p);
    };
    if constexpr (!DELTA)
      if (j0 == 0 && __any(live && brief)) {
        // the mean of dP, from the first key's on
        const float dp0 = __shfl(dp[0], lane % 32);
        float sum = 0.f, more = 0.f;
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) {
          const Points pt = points(r4);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = r4 * 4 + e;
            float th, d, inv;
            const float pr = weight(r, e, pt, th, d, inv);
            if (acc_row(r, h) < vis) sum += pr, more = fmaf(pr, dp[r] - dp0, more);
          }
        }
        sum += other_half(sum);
        more += other_half(more);
        if (brief && sum > 0.f) delta = dp0 + more / sum;
      }
#pragma unroll
    for (int r4 = 0; r4 < 4; ++r4) {
      const Points pt = points(r4);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = r4 * 4 + e;
        float th = 0.f, d = 0.f, inv = 0.f;
        const float pr = weight(r, e, pt, th, d, inv);
        if constexpr (DELTA) {
          gd = fmaf(pr, dp[r], gd);
        } else {
          float ds = pr * (dp[r] - delta);
          if constexpr (BIAS) {
            gs = fmaf(ds, d, gs);
            pt.add(e, ds * inv, gp);   // the slope is the column's own: at the end
          }
          if constexpr (CAP) ds = Cap<(WP > 1)>::slope(ds, th);
          s[r] = ds;
        }
      }
    }
    if (CAP && !BIAS && !DELTA && edge) {
      const int last = opaque(vis) - j0;
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if (acc_row(r, h) >= last) s[r] = 0.f;
    }
    if constexpr (DELTA) dsum[0] += gd;
    if constexpr (BIAS && !DELTA) v[0] += gp[0], v[1] += gp[1], v[2] += gp[2], v[3] += gs;
    if constexpr (!DELTA) TL::template outer<WP>(lk, s, dq[0], lane);
  };
  for (int j0 = kb; j0 < ke; j0 += ROWS * WV::STRIDE) {
    WV::sync();
    sk.store(st, lk);
    sv.store(st, lv);
    if (BIAS && st < ROWS) lp[st] = sp[0], lp[ROWS + st] = sp[1], lp[2 * ROWS + st] = sp[2];
    WV::sync();
    if (j0 + ROWS * WV::STRIDE < ke) fetch(j0 + ROWS * WV::STRIDE);

    tile(__any(j0 + ROWS > vis), j0);
  }
  float* slices = reinterpret_cast<float*>(lds);
  constexpr int slice = AREA;
  if constexpr (DELTA) {
    dsum[0] = (dsum[0] + other_half(dsum[0])) * norm.factor;
    if constexpr (MODE == kRows) join_values(slices, dsum);
    if (lead) part.delta[w.split * nrows + orow] = dsum[0];
    return;
  }
  if (lead && brief && w.split == 0) part.delta[orow] = delta;
  if constexpr (BIAS) {
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = (v[c] + other_half(v[c])) * norm.factor;
    if constexpr (MODE == kRows) join_values(slices, v);
    const float t = -kLn2 * slope, x[4] = {t * v[0], t * v[1], t * v[2], -v[3]};
    if (lead) store_f32<float, 4>(part.row + (w.split * nrows + orow) * 4, x);
  }
  if (!a.gq) return;   // the whole launch
#pragma unroll
  for (int b = 0; b < TL::DB; ++b)
#pragma unroll
    for (int r = 0; r < 16; ++r) dq[0][b][r] *= norm.factor * (CAP ? Cap<(WP > 1)>::kRest : 1.f);
  auto put = [&](size_t row, int d, const float* x) {
    const float y[4] = {x[0] * a.scale, x[1] * a.scale, x[2] * a.scale, x[3] * a.scale};
    if (part.splits == 1)
      store_f32<T, 4>(static_cast<T*>(a.gq) + row * a.D + d, y);
    else
      store_f32<float, 4>(part.o + (w.split * nrows + row) * a.D + d, y);
  };
  if constexpr (MODE == kRows) {
    join_waves(slices, slice, dq, a.D, [&](int c, int, int d, const float* x) {
      const int cc = w.tile * 32 + c, ii = cc / a.G;
      if (ii < w.lq) put((w.q0 + (size_t)ii) * a.hq + w.head * a.G + cc % a.G, d, x);
    });
  } else {
    each_piece(dq, h, a.D, [&](int, int d, const float* x) {
      if (live) put(orow, d, x);
    });
  }
}

// --------------------------------------------------- VJP: over key columns --

// What a row tile of packed queries carries besides q and g.
template <int ROWS, bool BIAS>
struct QueryTile {
  float ref[ROWS], factor[ROWS], delta[ROWS];
  int vis[ROWS];
  float pos[BIAS ? 3 : 1][BIAS ? ROWS : 4], slope[BIAS ? ROWS : 4];
};

template <class T, int DP, int MODE, bool BIAS, bool CAP>
__global__ __launch_bounds__(Waves<MODE>::TH, (waves_per_simd<T, DP, 1, MODE, BIAS>(2, 2, 2 + BIAS, 32)))
void attn_key_kernel(AttnArgs a, AttnPart part, int tiles) {
  using TL = Tile<T, DP, 1>;
  using WV = Waves<MODE>;
  constexpr int WP = kWeightParts<T, DP, MODE, true>;
  constexpr int ROWS = 32;
  constexpr int AREA = ROWS * TL::LD * TL::NP;   // LDS of one row tile
  __shared__ __align__(16) bf16 lds[WV::REGIONS * 2 * AREA];
  __shared__ __align__(16) QueryTile<ROWS, BIAS> lrow[WV::REGIONS];
  const Work w = find_work<true>(a, WV::COLS, 1, tiles, part.splits);
  if (!w.any) return;
  const int lane = threadIdx.x % 64, wv = uniform(threadIdx.x / 64), h = lane / 32, st = WV::stage_thread();
  const int j = w.tile * WV::COLS + (MODE == kCols ? wv * 32 : 0) + lane % 32;
  const bool live = j < w.lk;
  const size_t krow = w.k0 + j, nrows = (size_t)a.nq * a.hq;
  bf16 *lq = lds + WV::region() * 2 * AREA, *lg = lq + AREA;
  QueryTile<ROWS, BIAS>& lr = lrow[WV::region()];

  // Packed query rows [rb, re): those before the first that sees the block's
  // first key are left out.  A tile holds whole queries (all G heads) where
  // G <= 32, so that its rows lie the same way in every tile.
  const int jfirst = w.tile * WV::COLS, step = a.G <= ROWS ? ROWS / a.G * a.G : ROWS;
  const int i0 = a.causal && jfirst >= w.pre ? min(w.lq, max(0, jfirst - (w.lk - w.lq))) : 0;
  int rb, re;
  split_range((w.lq - i0) * a.G, step, part.splits, w.split, rb, re);
  rb += i0 * a.G, re += i0 * a.G;
  if (MODE == kRows) rb += wv * step;

  using ST = Stage<T, DP, 1, ROWS, WV::STAGE>;
  ST sq, sg;
  const uint32_t place = ST::place(st, a.D, a.G * a.D);
  float s_lse, s_delta, s_slope = 0.f, sp[3] = {0.f, 0.f, 0.f};
  int s_vis;
  const T* qbase = static_cast<const T*>(a.q) + (size_t)w.q0 * a.qs + (size_t)w.head * a.G * a.D;
  const T* gbase = static_cast<const T*>(a.g) + ((size_t)w.q0 * a.hq + (size_t)w.head * a.G) * a.D;
  const uint32_t qst = (uint32_t)a.qs * sizeof(T), gst = (uint32_t)(a.hq * a.D) * sizeof(T);
  const int row_bytes = a.G * a.D * (int)sizeof(T), head_bytes = a.D * (int)sizeof(T);
  uint32_t qoff[ST::N], goff[ST::N];
  int mi, mg;
  // rows of a tile that starts at head `rem` of a query
  auto lay_out = [&](int rem) {
    auto at = [&](int r, int& i, int& g) {
      i = a.G <= ROWS ? r / a.G : rem + r >= a.G;
      g = rem + r - i * a.G;
    };
#pragma unroll
    for (int n = 0; n < ST::N; ++n) {
      const int r = st / TL::CPR + n * ST::STEP;
      int i, g;
      at(r, i, g);
      const uint32_t p = r < step ? place : kNowhere;
      qoff[n] = p + i * qst + g * head_bytes;
      goff[n] = p + i * gst + g * head_bytes;
    }
    at(st % ROWS, mi, mg);   // the thread's row of the small values
  };
  lay_out(0);
  auto fetch = [&](int r0) {
    const int ib = r0 / a.G;
    if (a.G > ROWS) lay_out(r0 - ib * a.G);
    sq.load(make_rsrc(qbase + (size_t)ib * a.qs, reach(ib, w.lq, qst, row_bytes)), qoff);
    sg.load(make_rsrc(gbase + (size_t)ib * a.hq * a.D, reach(ib, w.lq, gst, row_bytes)), goff);
    if (st < ROWS) {
      const int i = ib + mi, head = w.head * a.G + mg;
      const bool on = st < step && r0 + st < re;
      const size_t orow = (size_t)(w.q0 + i) * a.hq + head;
      s_lse = on ? a.lse[orow] : -kInf;
      s_delta = on ? part.delta[orow] : 0.f;
      for (int s = 1; s < part.dsplits; ++s) s_delta += on ? part.delta[s * nrows + orow] : 0.f;
      s_vis = on ? visible(a, w, i) : 0;
      if constexpr (BIAS) {
#pragma unroll
        for (int k = 0; k < 3; ++k) sp[k] = on ? a.pos_q[3 * (size_t)(w.q0 + i) + k] : 0.f;
        s_slope = on ? a.slope[head] * kLog2e : 0.f;
      }
    }
  };
  if (rb < re) fetch(rb);

  typename TL::Cols kf, vf;
  f32x16 dk[1][TL::DB], dv[1][TL::DB];
  TL::load_cols(static_cast<const T*>(a.k) + (live ? krow * a.ks + (size_t)w.head * a.D : 0), live, a.D, h, kf);
  TL::load_cols(static_cast<const T*>(a.v) + (live ? krow * a.vs + (size_t)w.head * a.D : 0), live, a.D, h, vf);
#pragma unroll
  for (int b = 0; b < TL::DB; ++b) dk[0][b] = f32x16{}, dv[0][b] = f32x16{};
  float px = 0.f, py = 0.f, pz = 0.f;
  if (BIAS && live) px = a.pos_k[3 * krow], py = a.pos_k[3 * krow + 1], pz = a.pos_k[3 * krow + 2];
  const float c1 = a.scale * kLog2e;
  const Cap<(WP > 1)> cap(a.scale, a.cap);
  float gp[3] = {0.f, 0.f, 0.f};

  auto tile = [&](bool edge) {
    float gt[3] = {0.f, 0.f, 0.f};   // of this tile
    f32x16 s = TL::dot(lq, kf, lane);
    f32x16 dp = TL::dot(lg, vf, lane);
    if (edge) {
      const int jj = opaque(j);
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        const i32x4 vis = *reinterpret_cast<const i32x4*>(lr.vis + r4 * 8 + h * 4);
        const f32x4 delta = four(lr.delta + r4 * 8 + h * 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = r4 * 4 + e;
          if (!CAP && jj >= vis[e]) s[r] = -kInf;
          if (vis[e] == 1) dp[r] = delta[e];   // dS of a row with one key: 0
        }
      }
    }
#pragma unroll
    for (int r4 = 0; r4 < 4; ++r4) {
      const int rr = r4 * 8 + h * 4, pp = BIAS ? rr : 0;
      const f32x4 ref = four(lr.ref + rr), factor = four(lr.factor + rr), delta = four(lr.delta + rr);
      i32x4 vis;
      if constexpr (CAP && BIAS) vis = *reinterpret_cast<const i32x4*>(lr.vis + rr);
      const Points pt(px, py, pz, lr.pos[0] + pp, lr.pos[BIAS ? 1 : 0] + pp, lr.pos[BIAS ? 2 : 0] + pp);
      f32x4 sl;
      if constexpr (BIAS) sl = four(lr.slope + rr);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = r4 * 4 + e;
        float th = 0.f, x, inv;
        if constexpr (CAP) {
          x = cap.score(s[r], ref[e], th);
          if (BIAS && edge && j >= vis[e]) x = -kInf;
        } else {
          x = fmaf(s[r], c1, -ref[e]);
        }
        if constexpr (BIAS) {
          inv = inv_dist(pt.square(e));
          x = fmaf(-sl[e], dist_of<T>(pt.square(e), inv), x);
        }
        const float p = __builtin_amdgcn_exp2f(x) * factor[e];
        float ds = p * (dp[r] - delta[e]);
        if constexpr (BIAS) pt.add(e, ds * inv * sl[e], gt);
        if constexpr (CAP) ds = Cap<(WP > 1)>::slope(ds, th);
        s[r] = p;
        dp[r] = ds;
      }
    }
    if (CAP && !BIAS && edge) {
      const int jj = opaque(j);
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        const i32x4 vis = *reinterpret_cast<const i32x4*>(lr.vis + r4 * 8 + h * 4);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (jj >= vis[e]) s[r4 * 4 + e] = dp[r4 * 4 + e] = 0.f;
      }
    }
    if constexpr (BIAS) gp[0] += gt[0], gp[1] += gt[1], gp[2] += gt[2];
    TL::template outer<WP>(lg, s, dv[0], lane);
    TL::template outer<WP>(lq, dp, dk[0], lane);
  };
  for (int r0 = rb; r0 < re; r0 += step * WV::STRIDE) {
    WV::sync();
    sq.store(st, lq);
    sg.store(st, lg);
    if (st < ROWS) {
      const Norm norm(s_lse);
      lr.ref[st] = norm.ref;
      lr.factor[st] = norm.factor;
      lr.delta[st] = s_delta;
      lr.vis[st] = s_vis;
      if constexpr (BIAS) lr.pos[0][st] = sp[0], lr.pos[1][st] = sp[1], lr.pos[2][st] = sp[2], lr.slope[st] = s_slope;
    }
    WV::sync();
    // the tile's first row sees the least; absent rows see nothing
    const int s_least = step < ROWS || r0 + ROWS > re ? 0 : lr.vis[0];
    if (r0 + step * WV::STRIDE < re) fetch(r0 + step * WV::STRIDE);

    tile(__any(j >= s_least));
  }
  const size_t knum = (size_t)a.nk * a.hk;
  float* slices = reinterpret_cast<float*>(lds);
  constexpr int slice = AREA;
  if constexpr (BIAS) {
#pragma unroll
    for (int c = 0; c < 3; ++c) gp[c] += other_half(gp[c]);
    if constexpr (MODE == kRows) join_values(slices, gp);
    const float x[4] = {-kLn2 * gp[0], -kLn2 * gp[1], -kLn2 * gp[2], 0.f};
    if (live && h == 0 && (MODE != kRows || wv == 0))
      store_f32<float, 4>(part.col + (w.split * knum + krow * a.hk + w.head) * 4, x);
  }
  auto put = [&](T* out, float* split, float f, size_t row, int d, const float* x) {
    const float y[4] = {x[0] * f, x[1] * f, x[2] * f, x[3] * f};
    if (part.splits == 1)
      store_f32<T, 4>(out + row * a.D + d, y);
    else
      store_f32<float, 4>(split + (w.split * knum + row) * a.D + d, y);
  };
  auto write = [&](const f32x16 (&o)[1][TL::DB], void* out, float* split, float f) {
    if (!out) return;   // the whole launch
    if constexpr (MODE == kRows) {
      join_waves(slices, slice, o, a.D, [&](int c, int, int d, const float* x) {
        const int jj = w.tile * 32 + c;
        if (jj < w.lk) put(static_cast<T*>(out), split, f, (w.k0 + (size_t)jj) * a.hk + w.head, d, x);
      });
    } else {
      each_piece(o, h, a.D, [&](int, int d, const float* x) {
        if (live) put(static_cast<T*>(out), split, f, krow * a.hk + w.head, d, x);
      });
    }
  };
  write(dk, a.gk, part.o, a.scale * (CAP ? Cap<(WP > 1)>::kRest : 1.f));
  write(dv, a.gv, part.o2, 1.f);
}

// ---------------------------------------------------------------- launches --

template <class T, int DP, int HB, int MODE, bool BIAS, bool CAP>
void attn_launch_one(const AttnLaunch& l, const AttnArgs& a, const AttnPart& p, hipStream_t st) {
  const int splits = l.pass == kAttnDelta ? p.dsplits : p.splits;
  const int64_t cols = Waves<MODE>::COLS;
  const int tiles = (int)((l.pass == kAttnKey ? (int64_t)a.nk : (int64_t)a.nq * a.G) / cols + a.S);
  const int64_t units = (int64_t)(a.hk / HB) * splits;
  const int64_t blocks =
      8 % units == 0 ? 8 * ((tiles + 8 / units - 1) / (8 / units)) : units * tiles;
  const dim3 grid((unsigned)blocks), block(Waves<MODE>::TH);
  switch (l.pass) {
    case kAttnFwd: hipLaunchKernelGGL((attn_fwd_kernel<T, DP, HB, MODE, BIAS, CAP>), grid, block, 0, st, a, p, tiles); break;
    case kAttnDelta:
      if constexpr (sizeof(T) == 2 && BIAS && HB == 1)   // fp32: delta from out
        hipLaunchKernelGGL((attn_query_kernel<T, DP, MODE, BIAS, CAP, true>), grid, block, 0, st, a, p, tiles);
      break;
    case kAttnQuery:
      if constexpr (HB == 1)
        hipLaunchKernelGGL((attn_query_kernel<T, DP, MODE, BIAS, CAP, false>), grid, block, 0, st, a, p, tiles);
      break;
    default:
      if constexpr (HB == 1)
        hipLaunchKernelGGL((attn_key_kernel<T, DP, MODE, BIAS, CAP>), grid, block, 0, st, a, p, tiles);
      break;
  }
}

template <class T, int DP, int HB, bool BIAS>
void attn_launch_bias(const AttnLaunch& l, const AttnArgs& a, const AttnPart& p, hipStream_t st) {
  auto mode = [&](auto cap) {
    constexpr bool C = decltype(cap)::value;
    if constexpr (attn_cols_only(sizeof(T) == 2, DP)) {
      attn_launch_one<T, DP, HB, kCols, BIAS, C>(l, a, p, st);
    } else {
      switch (l.mode) {
        case kOne: attn_launch_one<T, DP, HB, kOne, BIAS, C>(l, a, p, st); break;
        case kCols: attn_launch_one<T, DP, HB, kCols, BIAS, C>(l, a, p, st); break;
        default: attn_launch_one<T, DP, HB, kRows, BIAS, C>(l, a, p, st); break;
      }
    }
  };
  a.cap > 0.f ? mode(std::integral_constant<bool, true>{}) : mode(std::integral_constant<bool, false>{});
}

template <class T, int DP>
void attn_launch(const AttnLaunch& l, const AttnArgs& a, const AttnPart& p, hipStream_t st) {
  if (!a.slope)
    attn_launch_bias<T, DP, 1, false>(l, a, p, st);
  else if (l.hb == 1)
    attn_launch_bias<T, DP, 1, true>(l, a, p, st);
  else if constexpr (attn_two_heads(sizeof(T) == 2, DP))
    attn_launch_bias<T, DP, 2, true>(l, a, p, st);
}

}  // namespace fc
