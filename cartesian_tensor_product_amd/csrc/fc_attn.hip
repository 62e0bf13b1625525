// Attention among the rows of each segment: how a call is cut into launches,
// and the reductions around the kernels of fc_attn_kernels.h.
//
// Splitting.  A column tile walks its whole row axis in one block when there
// are enough columns for the chip.  With few columns (single queries over
// many atoms) the walked axis is cut into `splits` parts, whose partial
// results go to the workspace and are joined in split order.
#include "fc_attn.h"

#include <algorithm>

#include "fc_reduce.h"
#include "fc_types.h"

namespace fc {
namespace {

// rows that belong to a segment; the others are left as they are
__device__ __forceinline__ bool in_segments(const int* off, int S, int n, int row) {
  return !off || (row >= max(0, off[0]) && row < min(n, off[S]));
}

// out = sum_s w_s o_s with w_s = exp(lse_s - lse); four elements per thread
template <class T>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a, AttnPart p) {
  const int per = a.D / 4;
  const size_t rows = (size_t)a.nq * a.hq, t = (size_t)blockIdx.x * 256 + threadIdx.x;
  const size_t row = t / per;
  const int d = (int)(t % per) * 4;
  if (row >= rows || !in_segments(a.seg_q, a.S, a.nq, (int)(row / a.hq))) return;
  float m = -__builtin_huge_valf();
  for (int s = 0; s < p.splits; ++s) m = fmaxf(m, p.lse[s * rows + row]);
  float o[4] = {0.f, 0.f, 0.f, 0.f}, sum = 0.f;
  if (m != -__builtin_huge_valf())
    for (int s = 0; s < p.splits; ++s) {
      const float w = __expf(p.lse[s * rows + row] - m);
      float x[4];
      load_f32<float, 4>(p.o + (s * rows + row) * a.D + d, x);
      sum += w;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = fmaf(w, x[i], o[i]);
    }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] *= inv;
  store_f32<T, 4>(static_cast<T*>(a.out) + row * a.D + d, o);
  if (d == 0) a.lse[row] = sum > 0.f ? m + __logf(sum) : m;
}

// out[row][.] = sum_s part[s][row][.] for rows of `width` elements
template <class T>
__global__ __launch_bounds__(256) void attn_sum_kernel(int n, int width, int S, int splits, const int* seg,
                                                       const float* __restrict__ part, T* __restrict__ out) {
  const size_t t = (size_t)blockIdx.x * 256 + threadIdx.x, total = (size_t)n * width, at = t * 4;
  if (at >= total || !in_segments(seg, S, n, (int)(at / width))) return;
  float x[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < splits; ++s) {
    float y[4];
    load_f32<float, 4>(part + s * total + at, y);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] += y[i];
  }
  store_f32<T, 4>(out + at, x);
}

// Position gradients of n rows from part0 [s0][n][h0][4] and, for rows that
// are keys as well, part1 [s1][n][h1][4] (heads and splits in order), and with
// `slope` the sums over a block's rows of part0's last component,
// [blocks][h0].  A block has `rows` rows with h0 threads side by side (x).
__global__ __launch_bounds__(256) void attn_row_kernel(int n, int S, const int* seg, int rows, int h0, int s0,
                                                       const float* __restrict__ part0, int h1, int s1,
                                                       const float* __restrict__ part1, float* __restrict__ pos,
                                                       float* __restrict__ slope) {
  __shared__ float lds[256][4];
  const int x = threadIdx.x, y = threadIdx.y, tid = y * blockDim.x + x;
  float sum = 0.f;
  const int lo = blockIdx.x * rows, hi = min(n, lo + rows);
  for (int i0 = lo; i0 < hi; i0 += blockDim.y) {
    const int i = i0 + y;
    const bool on = i < hi && in_segments(seg, S, n, i);
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (on && x < h0)
      for (int s = 0; s < s0; ++s) {
        float p[4];
        load_f32<float, 4>(part0 + (((size_t)s * n + i) * h0 + x) * 4, p);
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] += p[c];
      }
    sum += v[3];
    if (!pos) continue;   // the whole launch
    store_f32<float, 4>(lds[tid], v);
    __syncthreads();
    if (on && x < 3) {
      float t = 0.f;
      for (int h = 0; h < h0; ++h) t += lds[y * blockDim.x + h][x];
      for (int s = 0; part1 && s < s1; ++s)
        for (int h = 0; h < h1; ++h) t += part1[(((size_t)s * n + i) * h1 + h) * 4 + x];
      pos[3 * (size_t)i + x] = t;
    }
    __syncthreads();
  }
  if (!slope) return;
  lds[tid][0] = sum;
  __syncthreads();
  if (y != 0 || x >= h0) return;
  sum = 0.f;
  for (int k = 0; k < (int)blockDim.y; ++k) sum += lds[k * blockDim.x + x][0];
  slope[(size_t)blockIdx.x * h0 + x] = sum;
}

// ------------------------------------------------------------------- plans --

struct PassPlan {
  AttnMode mode;
  int hb, splits;
};

// `cols` columns and `rows` walked rows in all, over S segments; hk key heads.
//  * kCols (four waves with a row tile in common) loads least, and is taken
//    where its blocks of 128 columns, with the walk split in parts of 256 rows
//    at least, fill the chip (one block per CU).  With a block per CU without
//    it, only parts of 1024 rows are split off: partial results cost memory
//    traffic.
//  * Else four waves share the walk (kRows: four times the blocks; one segment
//    of 939 rows, one head of 64 in fp32, forward and VJP: 269 us as kCols with
//    8 blocks in one part against 70 us), also split in parts of 256 rows.
//  * Short walks (molecules): waves go alone (kOne).
//  * The key pass of wide bfloat16 heads (one wave per SIMD for its registers)
//    takes kRows also with many columns: with one wave, waiting for the three
//    others at every tile costs more than the shared loads save (packed batch of
//    8192 rows, 16 / 4 heads of 128: 215 us against 245 us).
PassPlan plan_pass(const AttnArgs& a, bool is_bf16, AttnPass pass, int64_t cols, int64_t rows) {
  PassPlan p;
  const int64_t mean = (cols + a.S - 1) / a.S, walk = rows / a.S;
  auto splits = [&](int64_t blocks, int64_t want, int64_t part) {
    return (int)std::clamp<int64_t>(std::min(want / std::max<int64_t>(1, blocks), walk / part), 1, 64);
  };
  p.hb = pass == kAttnFwd && a.slope && attn_two_heads(is_bf16, a.D) && a.hk % 2 == 0 && mean >= 32 ? 2 : 1;
  const int64_t units = (int64_t)a.S * (a.hk / p.hb);
  const int64_t wide = (mean + 127) / 128 * units, narrow = (mean + 31) / 32 * units;
  if (attn_cols_only(is_bf16, a.D)) {
    p.mode = kCols, p.splits = splits(wide, 512, wide < 256 ? 128 : 1024);
    return p;
  }
  if (walk < 128) {
    p.mode = mean >= 256 ? kCols : kOne, p.splits = 1;
    return p;
  }
  p.mode = kCols, p.splits = wide < 256 ? splits(wide, 512, 256) : splits(wide, 960, 1024);
  if (mean < 96 || wide * p.splits < 256) p.mode = kRows, p.splits = splits(narrow, 512, 256);
  if (pass == kAttnKey && is_bf16 && a.D > 64 && p.mode == kCols)
    p.mode = kRows, p.splits = splits(narrow, 4096, 2048);
  return p;
}

// rows of a block of attn_row_kernel: a thousand blocks at most
int rows_per_block(int n) { return std::max(32, (n + 1023) / 1024); }

struct Plan {
  PassPlan fwd, query, key;
  bool exact_delta;   // delta from the scores, not from the rounded out
  int slope_blocks;
  AttnPart pf, pd, pq, pk;
  float *row, *col, *slope;
  size_t bytes;
};

Plan make_plan(const AttnArgs& a, bool is_bf16, int op, void* ws) {
  Plan p{};
  const int64_t cq = (int64_t)a.nq * a.G;
  p.fwd = plan_pass(a, is_bf16, kAttnFwd, cq, a.nk);
  p.query = plan_pass(a, is_bf16, kAttnQuery, cq, a.nk);
  p.key = plan_pass(a, is_bf16, kAttnKey, a.nk, cq);
  // Position and slope gradients are fp32 outputs; with delta from a
  // bfloat16 out they would carry its rounding.
  p.exact_delta = is_bf16 && a.slope && (a.g_slope || a.g_pos_q || a.g_pos_k);
  size_t at = 0;
  auto take = [&](size_t floats) {
    float* q = reinterpret_cast<float*>(static_cast<char*>(ws) + at);
    at += (floats * sizeof(float) + 255) / 256 * 256;
    return q;
  };
  const size_t rq = (size_t)a.nq * a.hq, rk = (size_t)a.nk * a.hk;
  if (op == 0) {
    p.pf.splits = p.fwd.splits;
    if (p.fwd.splits > 1) {
      p.pf.o = take(p.fwd.splits * rq * a.D);
      p.pf.lse = take(p.fwd.splits * rq);
    }
  } else {
    AttnPart c{};
    c.exact = p.exact_delta;
    c.dsplits = p.exact_delta ? p.query.splits : 1;
    c.delta = take(c.dsplits * rq);
    if (a.slope) {
      c.row = take(p.query.splits * rq * 4);
      c.col = take(p.key.splits * rk * 4);
      p.slope_blocks = (a.nq + rows_per_block(a.nq) - 1) / rows_per_block(a.nq);
      p.slope = take((size_t)p.slope_blocks * a.hq);
    }
    const size_t nq = p.query.splits > 1 ? p.query.splits * rq * a.D : 0;
    const size_t nk = p.key.splits > 1 ? p.key.splits * rk * a.D : 0;
    // one after the other on the stream: the passes share this part
    float* o = take(std::max(nq, 2 * nk));
    p.pd = p.pq = p.pk = c;
    p.pq.splits = p.query.splits, p.pq.o = o;
    p.pk.splits = p.key.splits, p.pk.o = o, p.pk.o2 = o + nk;
  }
  p.bytes = at;
  return p;
}

template <class T>
void launch_dim(const AttnLaunch& l, const AttnArgs& a, const AttnPart& p, hipStream_t st) {
  if (a.D <= 16)
    attn_launch<T, 16>(l, a, p, st);
  else if (a.D <= 32)
    attn_launch<T, 32>(l, a, p, st);
  else if (a.D <= 64)
    attn_launch<T, 64>(l, a, p, st);
  else
    attn_launch<T, 128>(l, a, p, st);
}

void launch_pass(bool is_bf16, const AttnLaunch& l, const AttnArgs& a, const AttnPart& p, hipStream_t st) {
  is_bf16 ? launch_dim<bf16>(l, a, p, st) : launch_dim<float>(l, a, p, st);
}

unsigned blocks_of(size_t threads) { return (unsigned)((threads + 255) / 256); }

void sum_splits(bool is_bf16, int n, int width, int S, const int* seg, int splits, const float* part, void* out,
                hipStream_t st) {
  if (!out) return;
  const dim3 g(blocks_of((size_t)n * width / 4));
  if (is_bf16)
    hipLaunchKernelGGL(attn_sum_kernel<bf16>, g, dim3(256), 0, st, n, width, S, splits, seg, part,
                       static_cast<bf16*>(out));
  else
    hipLaunchKernelGGL(attn_sum_kernel<float>, g, dim3(256), 0, st, n, width, S, splits, seg, part,
                       static_cast<float*>(out));
}

}  // namespace

size_t attn_workspace_bytes(const AttnArgs& a, bool is_bf16, int op) {
  // the largest a call of this descriptor can need: with slopes and every
  // gradient, or without slopes (whose forward may split the keys further)
  AttnArgs b = a;
  static const float some = 0.f;
  b.slope = b.g_slope = nullptr;
  const size_t without = make_plan(b, is_bf16, op, nullptr).bytes;
  b.slope = &some;
  b.g_slope = const_cast<float*>(&some);
  return std::max(without, make_plan(b, is_bf16, op, nullptr).bytes);
}

void launch_attn_fwd(const AttnArgs& a, bool is_bf16, void* ws, hipStream_t st) {
  if (a.nq == 0) return;
  const Plan p = make_plan(a, is_bf16, 0, ws);
  launch_pass(is_bf16, {kAttnFwd, p.fwd.mode, p.fwd.hb}, a, p.pf, st);
  if (p.fwd.splits == 1) return;
  const dim3 g(blocks_of((size_t)a.nq * a.hq * (a.D / 4)));
  if (is_bf16)
    hipLaunchKernelGGL(attn_join_kernel<bf16>, g, dim3(256), 0, st, a, p.pf);
  else
    hipLaunchKernelGGL(attn_join_kernel<float>, g, dim3(256), 0, st, a, p.pf);
}

void launch_attn_vjp(const AttnArgs& a, bool is_bf16, void* ws, hipStream_t st) {
  const Plan p = make_plan(a, is_bf16, 1, ws);
  if (a.nq > 0) {   // also for the key pass alone: it leaves delta
    if (p.exact_delta) launch_pass(is_bf16, {kAttnDelta, p.query.mode, p.query.hb}, a, p.pd, st);
    launch_pass(is_bf16, {kAttnQuery, p.query.mode, p.query.hb}, a, p.pq, st);
    if (p.query.splits > 1)
      sum_splits(is_bf16, a.nq, a.hq * a.D, a.S, a.seg_q, p.query.splits, p.pq.o, a.gq, st);
  }
  if (a.nk > 0 && (a.gk || a.gv || a.g_pos_k || (a.g_pos_q && a.self_pos))) {
    launch_pass(is_bf16, {kAttnKey, p.key.mode, p.key.hb}, a, p.pk, st);
    if (p.key.splits > 1) {
      sum_splits(is_bf16, a.nk, a.hk * a.D, a.S, a.seg_k, p.key.splits, p.pk.o, a.gk, st);
      sum_splits(is_bf16, a.nk, a.hk * a.D, a.S, a.seg_k, p.key.splits, p.pk.o2, a.gv, st);
    }
  }
  auto rows = [&](int n, const int* seg, int h0, int s0, const float* p0, int h1, int s1, const float* p1, float* pos,
                  float* slope) {
    int x = 4;   // three threads at least write a row's position gradient
    while (x < h0) x <<= 1;
    const int run = rows_per_block(n);
    hipLaunchKernelGGL(attn_row_kernel, dim3((n + run - 1) / run), dim3(x, 256 / x), 0, st, n, a.S, seg, run, h0, s0, p0,
                       h1, s1, p1, pos, slope);
  };
  if ((a.g_pos_q || a.g_slope) && a.nq > 0)
    rows(a.nq, a.seg_q, a.hq, p.query.splits, p.pq.row, a.hk, p.key.splits, a.self_pos ? p.pk.col : nullptr, a.g_pos_q,
         a.g_slope ? p.slope : nullptr);
  if (a.g_pos_k && a.nk > 0)
    rows(a.nk, a.seg_k, a.hk, p.key.splits, p.pk.col, 0, 0, nullptr, a.g_pos_k, nullptr);
  if (a.g_slope) launch_column_sum(p.slope_blocks, a.hq, p.slope, a.g_slope, nullptr, st);
}

}  // namespace fc
