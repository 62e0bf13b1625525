// RMS norm of every query and key head with the rotation by position, for
// gfx950.  For a head row x of D elements at position p:
//   r = 1 / sqrt(mean x^2 + eps), y = gamma x r,
//   theta_t = <freq_t, p>, (o1, o2) = (y1 cos - y2 sin, y1 sin + y2 cos)
// for the R rotated pairs t; the other elements pass as y.  For the cotangent
// g of o, with gy = g rotated back and gg = gamma gy:
//   x_bar = r gg - x r^3 <gg, x> / D,  gamma_bar = sum gy x r,
//   theta_bar_t = sum_heads (gy2 y1 - gy1 y2),  p_bar = sum_t theta_bar_t freq_t.
//
// One pass over the data, bound by HBM.  A group of lanes holds a head row,
// each lane the same V pairs of every head, so that both members of a pair
// sit in one lane, and its cosines and sines are formed once per node and
// serve all of the node's heads.  The angle is formed in 64 bits and reduced
// to a turn there: at positions of 1e4 and more an fp32 angle has lost the
// digits that matter.
//
// Measured: forward, 131072 nodes, 4 + 4 heads of 32 in fp32, 63 us (4.3 TB/s);
// 40001 nodes, 16 + 4 heads of 128 in bfloat16, 91 us (4.5 TB/s) and VJP 155 us
// (4.0 TB/s).  A copy of that size runs at 5.1 TB/s.  The VJP loads a head row
// ahead (175 us without, 169 us with), stays within 128 registers so that all of
// its 1024 blocks are in flight (164 us) and adds up over lanes without LDS
// (156 us).
#include "fc_qk_rope.h"

#include <algorithm>

#include "fc_reduce.h"
#include "fc_types.h"

namespace fc {
namespace {

constexpr int kWaves = 4;      // of a block
constexpr int kVjpWaves = 4;   // per SIMD in the VJP: a thousand blocks at once

// Work of a lane: V pair slots from `slot`; P groups share a node.
struct Lane {
  int node0, head0, slot;
  bool live;
};

template <int V>
__device__ __forceinline__ Lane lane_of(int D, int group, int share) {
  const int lane = threadIdx.x % 64, w = threadIdx.x / 64;
  const int g = lane / group;
  Lane l;
  l.node0 = (blockIdx.x * kWaves + w) * (64 / (group * share)) + g / share;
  l.head0 = g % share;
  l.slot = (lane % group) * V;
  l.live = l.slot < D / 2;
  return l;
}

// element offsets of the two members of slots [s, s + V): halves (t, t + R)
// of the first 2R elements and halves of the rest, or neighbours
template <int V, bool INTER>
__device__ __forceinline__ void members(int s, int D, int R, int& a, int& b) {
  if constexpr (INTER) {
    a = 2 * s, b = 2 * s + V;
  } else {
    a = s < R ? s : R + s;
    b = s < R ? s + R : s + D / 2;
  }
}

// V pairs at row p into (x1, x2)
template <class T, int V, bool INTER>
__device__ __forceinline__ void load_pairs(const T* p, int a, int b, float* x1, float* x2) {
  if constexpr (INTER) {
    float x[2 * V];
    load_f32<T, V>(p + a, x);
    load_f32<T, V>(p + b, x + V);
#pragma unroll
    for (int i = 0; i < V; ++i) x1[i] = x[2 * i], x2[i] = x[2 * i + 1];
  } else {
    load_f32<T, V>(p + a, x1);
    load_f32<T, V>(p + b, x2);
  }
}

// the same in two steps: the pieces on their way, and their values
template <class T, int V>
struct Pieces {
  Pack<T, V> a, b;
  __device__ __forceinline__ void load(const T* p, int at_a, int at_b) {
    a = *reinterpret_cast<const Pack<T, V>*>(p + at_a);
    b = *reinterpret_cast<const Pack<T, V>*>(p + at_b);
  }
  template <bool INTER>
  __device__ __forceinline__ void get(float* x1, float* x2) const {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      x1[i] = static_cast<float>(INTER ? (2 * i < V ? a : b).e[2 * i % V] : a.e[i]);
      x2[i] = static_cast<float>(INTER ? (2 * i + 1 < V ? a : b).e[(2 * i + 1) % V] : b.e[i]);
    }
  }
};

template <class T, int V, bool INTER>
__device__ __forceinline__ void store_pairs(T* p, int a, int b, const float* x1, const float* x2) {
  if constexpr (INTER) {
    float x[2 * V];
#pragma unroll
    for (int i = 0; i < V; ++i) x[2 * i] = x1[i], x[2 * i + 1] = x2[i];
    store_f32<T, V>(p + a, x);
    store_f32<T, V>(p + b, x + V);
  } else {
    store_f32<T, V>(p + a, x1);
    store_f32<T, V>(p + b, x2);
  }
}

template <int V>
__device__ __forceinline__ void turn(const float (*freq)[3], const float* pos, float* c, float* s) {
  const double x = pos[0], y = pos[1], z = pos[2];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const double turns = (freq[i][0] * x + freq[i][1] * y + freq[i][2] * z) * 0.15915494309189533577;
    sincospif(2.f * static_cast<float>(turns - rint(turns)), &s[i], &c[i]);
  }
}

// v of the lane that the data-parallel control names (all lanes are active)
template <int CTRL>
__device__ __forceinline__ float moved(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}

// Sum over `group` neighbouring lanes (a power of two, the same for the wave).
// Up to 16 lanes by moves inside the vector unit: neighbours, pairs, then the
// mirrored half of 8 and of 16, whose lanes hold equal sums by then.  (Through
// LDS, as shuffles go, each step is a round trip that nothing else fills.)
__device__ __forceinline__ float group_sum(float v, int group) {
  if (group > 1) v += moved<0xb1>(v);
  if (group > 2) v += moved<0x4e>(v);
  if (group > 4) v += moved<0x141>(v);
  if (group > 8) v += moved<0x140>(v);
  if (group > 16) v += __shfl_xor(v, 16);
  if (group > 32) v += __shfl_xor(v, 32);
  return v;
}

template <int V>
__device__ __forceinline__ void load_freq(const QkRopeArgs& A, const Lane& l, float (*freq)[3]) {
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 3; ++j)   // pairs that only pass turn by nothing
      freq[i][j] = A.freq && l.slot + i < A.R ? A.freq[3 * (l.slot + i) + j] : 0.f;
}

// gamma of the lane's elements (ones when absent)
template <int V, bool INTER>
__device__ __forceinline__ void load_gamma(const float* gamma, const Lane& l, int a, int b, float* w1, float* w2) {
  if (gamma && l.live) {
    load_pairs<float, V, INTER>(gamma, a, b, w1, w2);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) w1[i] = w2[i] = 1.f;
  }
}

template <class T, int V, bool INTER>
__global__ __launch_bounds__(kWaves * 64) void qk_rope_fwd_kernel(QkRopeArgs A, int group, int share) {
  const Lane l = lane_of<V>(A.D, group, share);
  const int n = l.node0;
  // lanes without a node or slot take part in the sums with zeros
  const bool live = l.live && n < A.N;
  int a, b;
  members<V, INTER>(l.slot, A.D, A.R, a, b);
  float c[V], s[V];
  {
    float freq[V][3];
    load_freq<V>(A, l, freq);
    const float none[3] = {0.f, 0.f, 0.f};
    turn<V>(freq, A.pos && live ? A.pos + 3 * (size_t)n : none, c, s);
  }
  const float inv_d = 1.f / float(A.D);
  auto heads = [&](const T* x, int64_t stride, int H, const float* gamma, T* out) {
    float w1[V], w2[V];
    load_gamma<V, INTER>(gamma, l, a, b, w1, w2);
    for (int h0 = 0; h0 < H; h0 += share) {   // the same trips for the whole wave
      const int h = h0 + l.head0;
      const bool on = live && h < H;
      float x1[V] = {}, x2[V] = {};
      if (on) load_pairs<T, V, INTER>(x + (size_t)n * stride + (size_t)h * A.D, a, b, x1, x2);
      float q = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) q = fmaf(x1[i], x1[i], fmaf(x2[i], x2[i], q));
      const float r = 1.f / sqrtf(group_sum(q, group) * inv_d + A.eps);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float y1 = x1[i] * r * w1[i], y2 = x2[i] * r * w2[i];
        x1[i] = y1 * c[i] - y2 * s[i];
        x2[i] = y1 * s[i] + y2 * c[i];
      }
      if (on) store_pairs<T, V, INTER>(out + ((size_t)n * H + h) * A.D, a, b, x1, x2);
    }
  };
  heads(static_cast<const T*>(A.q), A.qs, A.hq, A.gamma_q, static_cast<T*>(A.q_out));
  heads(static_cast<const T*>(A.k), A.ks, A.hk, A.gamma_k, static_cast<T*>(A.k_out));
}

// Nodes in turn; a lane keeps the gamma gradients of its elements over all of
// its nodes and heads in registers.
template <class T, int V, bool INTER>
__global__ __launch_bounds__(kWaves * 64, kVjpWaves) void qk_rope_vjp_kernel(QkRopeArgs A, int group, int share) {
  __shared__ float lds[kWaves][2][kQkMaxDim];
  Lane l = lane_of<V>(A.D, group, share);
  int a, b;
  members<V, INTER>(l.slot, A.D, A.R, a, b);
  float freq[V][3];
  load_freq<V>(A, l, freq);
  const float inv_d = 1.f / float(A.D);
  const int stride_n = gridDim.x * kWaves * (64 / (group * share));
  float gam[2][2][V] = {};   // [queries, keys][member]
  const int first = l.node0 - (threadIdx.x % 64) / group / share;
  for (int n0 = first; n0 < A.N; n0 += stride_n) {   // the same trips for the whole wave
    const int n = n0 + l.node0 - first;
    const bool live = l.live && n < A.N;
    float c[V], s[V], th[V] = {};
    const float none[3] = {0.f, 0.f, 0.f};
    turn<V>(freq, A.pos && live ? A.pos + 3 * (size_t)n : none, c, s);
    auto heads = [&](const T* x, int64_t stride, int H, const float* gamma, const T* g, T* xb, float (*gm)[V]) {
      float w1[V], w2[V];
      load_gamma<V, INTER>(gamma, l, a, b, w1, w2);
      Pieces<T, V> px = {}, pg = {};
      auto fetch = [&](int h) {
        if (!live || h >= H) return;
        px.load(x + (size_t)n * stride + (size_t)h * A.D, a, b);
        pg.load(g + ((size_t)n * H + h) * A.D, a, b);
      };
      fetch(l.head0);
      for (int h0 = 0; h0 < H; h0 += share) {
        const int h = h0 + l.head0;
        const bool on = live && h < H;
        const size_t row = ((size_t)n * H + h) * A.D;
        float x1[V], x2[V], g1[V], g2[V];
        px.template get<INTER>(x1, x2);
        pg.template get<INTER>(g1, g2);
        if (!on)
#pragma unroll
          for (int i = 0; i < V; ++i) x1[i] = x2[i] = g1[i] = g2[i] = 0.f;
        fetch(h + share);
        float q = 0.f, d = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          q = fmaf(x1[i], x1[i], fmaf(x2[i], x2[i], q));
          const float t1 = g1[i] * c[i] + g2[i] * s[i], t2 = g2[i] * c[i] - g1[i] * s[i];
          g1[i] = t1;
          g2[i] = t2;
          d = fmaf(t1 * w1[i], x1[i], fmaf(t2 * w2[i], x2[i], d));
        }
        const float r = 1.f / sqrtf(group_sum(q, group) * inv_d + A.eps);
        const float k = group_sum(d, group) * inv_d * r * r;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float u1 = x1[i] * r, u2 = x2[i] * r;   // normalised
          gm[0][i] = fmaf(g1[i], u1, gm[0][i]);
          gm[1][i] = fmaf(g2[i], u2, gm[1][i]);
          th[i] += (g2[i] * u1) * w1[i] - (g1[i] * u2) * w2[i];
          x1[i] = r * (g1[i] * w1[i] - k * x1[i]);
          x2[i] = r * (g2[i] * w2[i] - k * x2[i]);
        }
        if (on && xb) store_pairs<T, V, INTER>(xb + row, a, b, x1, x2);
      }
    };
    heads(static_cast<const T*>(A.q), A.qs, A.hq, A.gamma_q, static_cast<const T*>(A.g_q), static_cast<T*>(A.q_grad),
          gam[0]);
    heads(static_cast<const T*>(A.k), A.ks, A.hk, A.gamma_k, static_cast<const T*>(A.g_k), static_cast<T*>(A.k_grad),
          gam[1]);
    if (A.pos_grad) {
      float p[3] = {0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 3; ++j) p[j] = fmaf(th[i], freq[i][j], p[j]);
#pragma unroll
      for (int j = 0; j < 3; ++j) p[j] = group_sum(p[j], group * share);
      if (n < A.N && (threadIdx.x % 64) % (group * share) == 0)
#pragma unroll
        for (int j = 0; j < 3; ++j) A.pos_grad[3 * (size_t)n + j] = p[j];
    }
  }
  if (!A.part) return;
  // lanes with the same slots: groups of the wave, then waves, then blocks
  const int w = threadIdx.x / 64;
#pragma unroll
  for (int m = 0; m < 2; ++m) {
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int i = 0; i < V; ++i)
        for (int o = group; o < 64; o <<= 1) gam[m][e][i] += __shfl_xor(gam[m][e][i], o);
    if (l.live && threadIdx.x % 64 < group) store_pairs<float, V, INTER>(lds[w][m], a, b, gam[m][0], gam[m][1]);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * A.D; i += kWaves * 64) {
    const int m = i / A.D, e = i % A.D;
    float t = 0.f;
#pragma unroll
    for (int v = 0; v < kWaves; ++v) t += lds[v][m][e];
    A.part[((size_t)m * gridDim.x + blockIdx.x) * A.D + e] = t;
  }
}

// Pairs per lane: 16-byte pieces where the halves and the rows allow them, in
// the VJP four pairs at most.
int pairs_per_lane(const QkRopeArgs& a, bool vjp) {
  const int e = a.bf16 ? 2 : 4, full = vjp ? 4 : 16 / e;
  auto fits = [&](int v) {
    auto on = [&](const void* p) { return reinterpret_cast<uintptr_t>(p) % (v * e) == 0; };
    auto on4 = [&](const void* p) { return reinterpret_cast<uintptr_t>(p) % (v * 4) == 0; };
    return (a.D / 2) % v == 0 && (a.interleaved || a.R % v == 0) && a.qs % v == 0 && a.ks % v == 0 && on(a.q) &&
           on(a.k) && on(a.q_out) && on(a.k_out) && on(a.g_q) && on(a.g_k) && on(a.q_grad) && on(a.k_grad) &&
           on4(a.gamma_q) && on4(a.gamma_k);
  };
  return fits(full) ? full : fits(4) ? 4 : fits(2) ? 2 : 1;
}

struct Shape {
  int vec, group, share;   // lanes of a row, groups of a node
  int waves;               // waves that give every node one turn
};

Shape shape_of(const QkRopeArgs& a, int vec) {
  Shape s{vec, 1, 1, 0};
  while (s.group * vec < a.D / 2) s.group <<= 1;
  // nodes of few: the heads of a node spread over the wave's groups, until
  // every SIMD has about four waves
  const int most = std::max(a.hq, a.hk);
  auto waves = [&](int share) { return (int)(((int64_t)a.N * s.group * share + 63) / 64); };
  while (s.group * s.share < 64 && s.share < most && waves(s.share) < 4096) s.share <<= 1;
  s.waves = waves(s.share);
  return s;
}

template <int MOST, class F>
void dispatch(const QkRopeArgs& a, int vec, F&& f) {
  auto inter = [&](auto t, auto v) {
    a.interleaved ? f(t, v, std::integral_constant<bool, true>{}) : f(t, v, std::integral_constant<bool, false>{});
  };
  auto type = [&](auto v) {
    if constexpr (decltype(v)::value <= 4) {
      a.bf16 ? inter(bf16{}, v) : inter(float{}, v);
    } else {
      inter(bf16{}, v);   // eight pairs are 16 bytes of bfloat16
    }
  };
  switch (vec) {
    case 8:
      if constexpr (MOST == 8) type(std::integral_constant<int, 8>{});
      break;
    case 4: type(std::integral_constant<int, 4>{}); break;
    case 2: type(std::integral_constant<int, 2>{}); break;
    default: type(std::integral_constant<int, 1>{}); break;
  }
}

}  // namespace

// The lane layout depends on alignment, so the bound holds for every layout.
int qk_rope_vjp_blocks(const QkRopeArgs& a) {
  const int64_t groups = ((int64_t)a.N * 64 + 63) / 64;
  return (int)std::min<int64_t>(1024, (groups + kWaves - 1) / kWaves);
}

void launch_qk_rope_fwd(const QkRopeArgs& a, hipStream_t st) {
  const int vec = pairs_per_lane(a, false);
  const Shape s = shape_of(a, vec);
  dispatch<8>(a, vec, [&](auto t, auto v, auto inter) {
    hipLaunchKernelGGL((qk_rope_fwd_kernel<decltype(t), decltype(v)::value, decltype(inter)::value>),
                       dim3((s.waves + kWaves - 1) / kWaves), dim3(kWaves * 64), 0, st, a, s.group, s.share);
  });
}

void launch_qk_rope_vjp(const QkRopeArgs& a, float* gamma_q_grad, float* gamma_k_grad, hipStream_t st) {
  const int vec = pairs_per_lane(a, true);
  const Shape s = shape_of(a, vec);
  const int blocks = std::min((s.waves + kWaves - 1) / kWaves, qk_rope_vjp_blocks(a));
  dispatch<4>(a, vec, [&](auto t, auto v, auto inter) {
    hipLaunchKernelGGL((qk_rope_vjp_kernel<decltype(t), decltype(v)::value, decltype(inter)::value>), dim3(blocks),
                       dim3(kWaves * 64), 0, st, a, s.group, s.share);
  });
  launch_column_sum(blocks, a.D, a.part, gamma_q_grad, gamma_k_grad, st);
}

}  // namespace fc
