// Scaled lookup of table rows (species, tokens) and its gradient for gfx950:
//   out[n][c]  = scale table[id_n][c],
//   grad[r][c] = scale sum_{n : id_n = r} g[n][c],
// ids outside [0, R) are padding: a zero row, no gradient.
//
// Lookup: 16-byte pieces, a lane each; bound by the write of out (300000 tokens,
// 95 rows of 128 in fp32: 28 us, 5.5 TB/s; one call of 1000 tokens 2.4 us).
//
// Gradient: sums over tokens of one row in a fixed order, without
// floating-point atomics, from a stable sort of the ids.
//  * Tables of up to 255 rows (species): a block sorts 1024 neighbouring tokens
//    and sums them row by row; a second kernel adds up the blocks.  300000
//    tokens, 95 rows of 128 in fp32: 51 and 5 us; bound by the read of g (3 TB/s)
//    behind each block's own sort.
//  * Larger ones: a radix sort of all ids gives the tokens of each row as one run
//    of the sorted order, cut into chunks of equal length whatever the runs are,
//    so that one very frequent row costs no more than many rare ones.  A group of
//    lanes walks its chunk, adds the tokens' rows in fp32 and writes a row when
//    its run ends; the runs cut by a chunk edge go to partial sums (at most two
//    per chunk), which the last kernel adds in chunk order.  That kernel also
//    writes the zeros of rows without a token.  65536 tokens, 50000 rows of 512 in
//    bfloat16: two sorting passes 32 us, the sums 30 and the join, which writes
//    most of the 102 MB table, 20 (5 TB/s).
// Lookup and gradient with 255 rows and, all ids sorted, with 256: 300000 tokens
// of 128 channels 94 and 115 us in fp32, 52 and 94 us in bfloat16; 4096 tokens 17
// and 30 us.
#include "fc_embed.h"

#include <algorithm>
#include <type_traits>

#include "fc_types.h"

namespace fc {
namespace {

constexpr int kSortThreads = 256, kSortRounds = 4, kSortItems = kSortThreads * kSortRounds;
constexpr int kSortWaves = kSortThreads / 64;

template <class T, int V>
__global__ __launch_bounds__(256) void embed_fwd_kernel(int N, int R, int C, float scale, const T* __restrict__ table,
                                                        const int* __restrict__ ids, T* __restrict__ out) {
  for (int n = blockIdx.x * blockDim.y + threadIdx.y; n < N; n += gridDim.x * blockDim.y) {
    const int id = ids[n];
    const bool real = id >= 0 && id < R;
    const T* src = table + (size_t)(real ? id : 0) * C;
    T* dst = out + (size_t)n * C;
    for (int c = threadIdx.x * V; c < C; c += blockDim.x * V) {
      float x[V];
      load_f32<T, V>(src + c, x);
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = real ? x[i] * scale : 0.f;
      store_f32<T, V>(dst + c, x);
    }
  }
}

// ---------------------------------------------------------------- the sort --

// ids as sort keys: padding sorts behind the last row
__device__ __forceinline__ int key_of(int id, int R) { return id >= 0 && id < R ? id : R; }

// counts of one digit per block, hist[digit][block]
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(int N, int R, int shift, int ndig, bool first_pass,
                                                                  const int* __restrict__ keys,
                                                                  int* __restrict__ hist) {
  __shared__ int cnt[256];
  const int t = threadIdx.x;
  cnt[t] = 0;
  __syncthreads();
  const int base = blockIdx.x * kSortItems;
#pragma unroll
  for (int i = 0; i < kSortRounds; ++i) {
    const int n = base + i * kSortThreads + t;
    if (n < N) {
      const int k = first_pass ? key_of(keys[n], R) : keys[n];
      atomicAdd(&cnt[(k >> shift) & (ndig - 1)], 1);   // integer counts: no order
    }
  }
  __syncthreads();
  if (t < ndig) hist[(size_t)t * gridDim.x + blockIdx.x] = cnt[t];
}

// exclusive scan over the blocks of one digit (one block per digit); the
// grid also clears the run bounds of R rows (0 but in the first pass)
__global__ __launch_bounds__(256) void sort_scan_kernel(int nblk, int* __restrict__ hist, int* __restrict__ total,
                                                        int R, int* __restrict__ first, int* __restrict__ last) {
  __shared__ int sums[4];
  const int t = threadIdx.x, lane = t % 64, w = t / 64;
  int* h = hist + (size_t)blockIdx.x * nblk;
  int carry = 0;
  for (int b0 = 0; b0 < nblk; b0 += 256) {
    const int v = b0 + t < nblk ? h[b0 + t] : 0;
    int s = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(s, o);
      if (lane >= o) s += u;
    }
    if (lane == 63) sums[w] = s;
    __syncthreads();
    int before = carry, all = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < w) before += sums[i];
      all += sums[i];
    }
    if (b0 + t < nblk) h[b0 + t] = before + s - v;
    carry += all;
    __syncthreads();
  }
  if (t == 0) total[blockIdx.x] = carry;
  for (int r = blockIdx.x * 256 + t; r < R; r += gridDim.x * 256) first[r] = last[r] = 0;
}

// Rank of the lane's digit d (bits wide; lanes out of `in` have none) among the
// keys that the wave has seen: those counted in cnt, and those of lower lanes,
// found by one ballot per bit.  Counts them.
__device__ __forceinline__ int rank_of(int d, bool in, int bits, int lane, int* cnt) {
  unsigned long long peers = __ballot(in);
  for (int b = 0; b < bits; ++b) {
    const bool set = (d >> b) & 1;
    const unsigned long long m = __ballot(in && set);
    peers &= set ? m : ~m;
  }
  const int rank = in ? cnt[d] + __popcll(peers & ((1ull << lane) - 1)) : 0;
  // every lane has read its count before the last peer adds the group
  // (a wave's LDS accesses are served in order; the fences hold the compiler)
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  if (in && (peers >> lane) == 1ull) cnt[d] = rank + 1;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  return rank;
}

// Sum over the lower lanes of the 256 threads' values v (all threads of the
// block call it; those from 256 on add nothing)
__device__ __forceinline__ int sum_before(int v, int t, int* sums) {
  const int lane = t % 64, w = t / 64;
  int s = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(s, o);
    if (lane >= o) s += u;
  }
  if (lane == 63 && w < 4) sums[w] = s;
  __syncthreads();
  int run = s - v;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < w) run += sums[i];
  return run;
}

// Stable scatter: a wave takes 64 neighbouring keys at a time
// and counts on from its own earlier keys; waves and blocks follow in order.
__global__ __launch_bounds__(kSortThreads) void sort_scatter_kernel(int N, int R, int shift, int bits, bool first_pass,
                                                                    const int* __restrict__ keys,
                                                                    const int* __restrict__ ord,
                                                                    const int* __restrict__ hist,
                                                                    const int* __restrict__ total,
                                                                    int* __restrict__ keys_out,
                                                                    int* __restrict__ ord_out) {
  __shared__ int cnt[kSortWaves][256];
  __shared__ int sums[kSortWaves];
  const int t = threadIdx.x, lane = t % 64, w = t / 64, ndig = 1 << bits;
#pragma unroll
  for (int i = 0; i < kSortWaves; ++i) cnt[i][t] = 0;
  const int base = blockIdx.x * kSortItems + w * (kSortItems / kSortWaves);
  int key[kSortRounds], rank[kSortRounds];
#pragma unroll
  for (int i = 0; i < kSortRounds; ++i) {
    const int n = base + i * 64 + lane;
    key[i] = n < N ? (first_pass ? key_of(keys[n], R) : keys[n]) : 0;
  }
  const int digits = t < ndig ? total[t] : 0;
  const int before = t < ndig ? hist[(size_t)t * gridDim.x + blockIdx.x] : 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSortRounds; ++i) {
    const bool in = base + i * 64 + lane < N;
    rank[i] = rank_of((key[i] >> shift) & (ndig - 1), in, bits, lane, cnt[w]);
  }
  __syncthreads();
  {  // digit t: first position = digits before + blocks before + waves before
    int run = sum_before(digits, t, sums) + before;
#pragma unroll
    for (int i = 0; i < kSortWaves; ++i) {
      const int c = cnt[i][t];
      cnt[i][t] = run;
      run += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSortRounds; ++i) {
    const int n = base + i * 64 + lane;
    if (n >= N) continue;
    const int p = cnt[w][(key[i] >> shift) & (ndig - 1)] + rank[i];
    keys_out[p] = key[i];
    ord_out[p] = first_pass ? n : ord[n];
  }
}

// The whole sort of at most kSmall ids in one block, in LDS; the other blocks
// clear the run bounds.  Three launches in all instead of five or eight (lookup
// and gradient over 5000 rows of 128 channels: 4096 tokens 35 us, 4097 tokens,
// sorted by the kernels above, 46 us).
constexpr int kSmall = 4096, kSmallThreads = 1024;
__global__ __launch_bounds__(kSmallThreads) void sort_small_kernel(int N, int R, int bits, int passes,
                                                                   const int* __restrict__ ids,
                                                                   int* __restrict__ keys_out,
                                                                   int* __restrict__ ord_out, int* __restrict__ first,
                                                                   int* __restrict__ last) {
  constexpr int W = kSmallThreads / 64, ROUNDS = kSmall / kSmallThreads;
  __shared__ int key[2][kSmall], ord[2][kSmall], cnt[W][256], sums[4];
  const int t = threadIdx.x, lane = t % 64, w = t / 64, ndig = 1 << bits;
  if (blockIdx.x > 0) {
    for (int r = (blockIdx.x - 1) * kSmallThreads + t; r < R; r += (gridDim.x - 1) * kSmallThreads)
      first[r] = last[r] = 0;
    return;
  }
  for (int n = t; n < N; n += kSmallThreads) key[0][n] = key_of(ids[n], R), ord[0][n] = n;
  for (int s = 0; s < passes; ++s) {
    const int *k = key[s & 1], *o = ord[s & 1], shift = s * bits;
    for (int i = t; i < W * 256; i += kSmallThreads) cnt[i / 256][i % 256] = 0;
    __syncthreads();
    const int base = w * (kSmall / W) + lane;
    int rank[ROUNDS];
#pragma unroll
    for (int i = 0; i < ROUNDS; ++i) {
      const int n = base + i * 64;
      rank[i] = rank_of((k[min(n, N - 1)] >> shift) & (ndig - 1), n < N, bits, lane, cnt[w]);
    }
    __syncthreads();
    int all = 0;
    if (t < 256)
      for (int i = 0; i < W; ++i) all += cnt[i][t];
    int run = sum_before(all, t, sums);
    if (t < 256)
      for (int i = 0; i < W; ++i) {
        const int c = cnt[i][t];
        cnt[i][t] = run;
        run += c;
      }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ROUNDS; ++i) {
      const int n = base + i * 64;
      if (n >= N) continue;
      const int p = cnt[w][(k[n] >> shift) & (ndig - 1)] + rank[i];
      key[(s + 1) & 1][p] = k[n];
      ord[(s + 1) & 1][p] = o[n];
    }
    __syncthreads();
  }
  for (int n = t; n < N; n += kSmallThreads) keys_out[n] = key[passes & 1][n], ord_out[n] = ord[passes & 1][n];
}

// ---------------------------------------------------------------- the sums --

// One group of `group` lanes per (chunk, channel slice); lane i of the group
// holds V channels.  Shorter chunks (32 tokens for 64) leave its time as it is
// and lengthen the join (9 to 13 us, 300000
// tokens over 95 rows).  part[chunk][2][C]: the sum of the run that begins at or
// before the chunk's first token and does not end inside it alone (slot 0),
// and of the run that begins inside and continues behind the chunk (slot 1).
template <class T, int V>
__global__ __launch_bounds__(256) void embed_sum_kernel(int N, int R, int C, int chunk, int chunks, int group,
                                                        int slices, float scale, const int* __restrict__ key,
                                                        const int* __restrict__ ord, const T* __restrict__ g,
                                                        float* __restrict__ grad, float* __restrict__ part,
                                                        int* __restrict__ first, int* __restrict__ last) {
  const int per = 256 / group;
  const long long item = (long long)blockIdx.x * per + threadIdx.x / group;
  const int ch = int(item / slices), c = (int(item % slices) * group + threadIdx.x % group) * V;
  if (ch >= chunks) return;
  const bool live = c < C, lead = c == 0;
  const int p0 = ch * chunk, p1 = min(N, p0 + chunk);
  const int before = p0 > 0 ? key[p0 - 1] : -1, after = p1 < N ? key[p1] : -1;
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
  int cur = key[p0], begin = p0;
  auto flush = [&](int end) {
    // the run [begin, end) of row cur inside this chunk
    const bool from_before = begin == p0 && before == cur, goes_on = end == p1 && after == cur;
    if (lead) {
      if (!from_before) first[cur] = begin;
      if (!goes_on) last[cur] = end;
    }
    if (!live) return;
    float* dst;
    float f = 1.f;
    if (!from_before && !goes_on) {
      dst = grad + (size_t)cur * C;
      f = scale;
    } else {
      dst = part + ((size_t)ch * 2 + (from_before || begin == p0 ? 0 : 1)) * C;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] *= f;
    store_f32<float, V>(dst + c, acc);
  };
  // U rows in flight; their keys and places are read a batch ahead, by one
  // lane each where a group has that many
  constexpr int U = 16;
  const int gl = threadIdx.x % group, g0 = threadIdx.x % 64 - gl;
  const bool shared = group >= U;
  int kn = 0, on = 0;
  auto ahead = [&](int p) {
    const int q = min(p + gl % U, p1 - 1);
    kn = key[q];
    on = ord[q];
  };
  if (shared) ahead(p0);
  for (int p = p0; p < p1; p += U) {
    int k[U];
    Pack<T, V> x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int q = min(p + u, p1 - 1);
      k[u] = shared ? __shfl(kn, g0 + u) : key[q];
      const int o = shared ? __shfl(on, g0 + u) : ord[q];
      if (live && k[u] < R) x[u] = *reinterpret_cast<const Pack<T, V>*>(g + (size_t)o * C + c);
    }
    if (shared && p + U < p1) ahead(p + U);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (p + u >= p1) break;
      if (k[u] != cur) {
        flush(p + u);
        cur = k[u];
        begin = p + u;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.f;
      }
      if (cur >= R) return;   // padding is sorted last
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] += static_cast<float>(x[u].e[i]);
    }
  }
  flush(p1);
}

// Rows whose run is cut by chunk edges, and rows without a token.  A wave
// takes RW rows, 64 / group of them side by side (lookup and gradient of 49
// tokens over 47725 rows of 24 channels: 31 us; 50 us with one row at a time).
// The rows of a block lie a grid apart, so that neighbouring frequent rows
// (tables are often ordered by frequency) fall to different blocks.  Rows of
// more than kLong pieces are left to the whole block, whose waves take pieces in
// turn and add up in wave order.  gridDim.y blocks share the channels.
constexpr int kLong = 16;
template <int W, int RW, int V>
__global__ __launch_bounds__(W * 64) void embed_join_kernel(int R, int C, int chunk, int group, float scale,
                                                            const int* __restrict__ first,
                                                            const int* __restrict__ last,
                                                            const float* __restrict__ part, float* __restrict__ grad) {
  // rows of the block: RW per wave, or one for all of a block of RW = 1
  constexpr int ROWS = RW == 1 ? 1 : W * RW;
  __shared__ float sum[W][64 * V];
  __shared__ int bound[2][ROWS];
  const int w = threadIdx.x / 64, lane = threadIdx.x % 64;
  auto row = [&](int i) { return (int)(blockIdx.x + i * gridDim.x); };
  const int rows = (R - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;   // at most ROWS
  auto is_long = [&](int f, int l) { return l > f && (l - 1) / chunk - f / chunk >= kLong; };
  bool own_long = false;
  if (threadIdx.x < rows) {
    const int f = first[row(threadIdx.x)], l = last[row(threadIdx.x)];
    bound[0][threadIdx.x] = f, bound[1][threadIdx.x] = l;
    own_long = is_long(f, l);
  }
  const bool any_long = __syncthreads_or(own_long);
  // piece of the run of chunks a..b: slot 1 of a unless the run begins there
  auto slot = [&](int f, int ch) { return part + ((size_t)ch * 2 + (ch * chunk < f ? 1 : 0)) * C; };
  for (int i = w * RW + lane / group; i < min(rows, (w + 1) * RW); i += 64 / group) {
    const int f = bound[0][i], l = bound[1][i], a = f / chunk, b = (l - 1) / chunk;
    if (is_long(f, l) || (l > f && a == b)) continue;
    for (int c = (blockIdx.y * group + lane % group) * V; c < C; c += gridDim.y * group * V) {
      float acc[V] = {};
      for (int ch = a; l > f && ch <= b; ++ch) {
        float x[V];
        load_f32<float, V>(slot(f, ch) + c, x);
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] += x[e];
      }
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] *= scale;
      store_f32<float, V>(grad + (size_t)row(i) * C + c, acc);
    }
  }
  if (!any_long) return;   // the same for the whole block
  for (int i = 0; i < rows; ++i) {
    const int f = bound[0][i], l = bound[1][i], a = f / chunk, b = (l - 1) / chunk;
    if (l <= f || b - a < kLong) continue;
    for (int c0 = blockIdx.y * 64 * V; c0 < C; c0 += gridDim.y * 64 * V) {
      const int c = c0 + lane * V;
      float acc[V] = {};
      if (c < C) {
#pragma unroll 8
        for (int ch = a + w; ch <= b; ch += W) {
          float x[V];
          load_f32<float, V>(slot(f, ch) + c, x);
#pragma unroll
          for (int e = 0; e < V; ++e) acc[e] += x[e];
        }
      }
#pragma unroll
      for (int e = 0; e < V; ++e) sum[w][lane * V + e] = acc[e];
      __syncthreads();
      if (w == 0 && c < C) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float t = 0.f;
          for (int j = 0; j < W; ++j) t += sum[j][lane * V + e];
          acc[e] = t * scale;
        }
        store_f32<float, V>(grad + (size_t)row(i) * C + c, acc);
      }
      __syncthreads();
    }
  }
}

// ----------------------------------------------------------- tables of few rows --

// A table of few rows (species): a block sorts a window of kWindow tokens in
// LDS, sums the runs of that order and writes its sum of every row,
// part[window][R][C]; the next kernel adds the windows in order.  Each group of
// lanes walks `per` tokens; runs that go on over groups meet in LDS.  The rows of
// g are read window by window, not over all tokens row by row.
constexpr int kWindow = 1024, kFewRows = 255;   // keys 0..255: one digit
template <class T, int V>
__global__ __launch_bounds__(kWindow) void embed_window_kernel(int N, int R, int C, int group, int per,
                                                               const int* __restrict__ ids, const T* __restrict__ g,
                                                               float* __restrict__ part) {
  constexpr int W = kWindow / 64;
  __shared__ int cnt[W][256], start[256], sums[4], key[kWindow], ord[kWindow];
  // sums of a group's first run where it began before (0), and of its last where
  // it goes on (1)
  __shared__ __align__(32) float edge[2][kWindow * V];
  const int t = threadIdx.x, lane = t % 64, w = t / 64;
  for (int i = t; i < W * 256; i += kWindow) cnt[i / 256][i % 256] = 0;
  const int n = blockIdx.x * kWindow + t;
  const int k = n < N ? key_of(ids[n], R) : R;   // below 256
  __syncthreads();
  const int rank = rank_of(k, true, 8, lane, cnt[w]);
  __syncthreads();
  int all = 0;
  if (t < 256)
    for (int i = 0; i < W; ++i) all += cnt[i][t];
  int run = sum_before(all, t, sums);
  if (t < 256) {
    start[t] = run;
    for (int i = 0; i < W; ++i) {
      const int c = cnt[i][t];
      cnt[i][t] = run;
      run += c;
    }
  }
  __syncthreads();
  const int place = cnt[w][k] + rank;
  key[place] = k;
  ord[place] = n;
  __syncthreads();
  const int real = start[R];   // padding is sorted last
  const int gi = t / group, c = (blockIdx.y * group + t % group) * V;
  const int p0 = gi * per, p1 = min(p0 + per, real);
  const bool on = c < C;
  float* out = part + (size_t)blockIdx.x * R * C + c;
  float acc[V] = {};
  int cur = 0;
  bool goes_on = false;
  if (p0 < p1 && on) {
    cur = key[p0];
    bool before = p0 > 0 && key[p0 - 1] == cur;
    auto put = [&](float* dst) { store_f32<float, V>(dst, acc); };
    constexpr int U = 16;
    for (int p = p0; p < p1; p += U) {
      Pack<T, V> x[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        x[u] = *reinterpret_cast<const Pack<T, V>*>(g + (size_t)ord[min(p + u, p1 - 1)] * C + c);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (p + u >= p1) break;
        const int next = key[p + u];
        if (next != cur) {
          put(before ? edge[0] + t * V : out + (size_t)cur * C);
          before = false;
          cur = next;
#pragma unroll
          for (int e = 0; e < V; ++e) acc[e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] += static_cast<float>(x[u].e[e]);
      }
    }
    goes_on = p1 < real && key[p1] == cur;
    put(before ? edge[0] + t * V : goes_on ? edge[1] + t * V : out + (size_t)cur * C);
    goes_on &= !before;
  }
  __syncthreads();
  if (goes_on) {
    for (int h = gi + 1; h * per < real && key[h * per] == cur; ++h) {
      float x[V];
      load_f32<float, V>(edge[0] + (t + (h - gi) * group) * V, x);
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] += x[e];
    }
    store_f32<float, V>(out + (size_t)cur * C, acc);
  }
  if (!on) return;
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] = 0.f;
  for (int r = gi; r < R; r += kWindow / group)
    if (start[r] == start[r + 1]) store_f32<float, V>(out + (size_t)r * C, acc);
}

// grad[i] = scale sum_b part[b][i]: a block of 16 waves for 64 columns
__global__ __launch_bounds__(1024) void embed_window_join_kernel(int windows, size_t n, float scale,
                                                                 const float* __restrict__ part,
                                                                 float* __restrict__ grad) {
  __shared__ float sum[16][64];
  const int lane = threadIdx.x % 64, w = threadIdx.x / 64;
  const size_t i = (size_t)blockIdx.x * 64 + lane;
  float acc = 0.f;
  if (i < n)
#pragma unroll 8
    for (int b = w; b < windows; b += 16) acc += part[b * n + i];
  sum[w][lane] = acc;
  __syncthreads();
  if (w > 0 || i >= n) return;
  for (int j = 1; j < 16; ++j) acc += sum[j][lane];
  grad[i] = acc * scale;
}

int pow2_at_least(int n) {
  int p = 1;
  while (p < n) p <<= 1;
  return p;
}

// channels per lane: 16 bytes of the element type where rows allow it
int vec_of(int C, bool bf16, bool aligned) {
  int v = aligned ? bf16 ? 8 : 4 : 1;
  while (C % v != 0) v >>= 1;
  return v;
}

template <class F>
void dispatch(bool is_bf16, int vec, F&& f) {
  auto type = [&](auto v) { is_bf16 ? f(bf16{}, v) : f(float{}, v); };
  switch (vec) {
    case 8: f(bf16{}, std::integral_constant<int, 8>{}); break;
    case 4: type(std::integral_constant<int, 4>{}); break;
    case 2: type(std::integral_constant<int, 2>{}); break;
    default: type(std::integral_constant<int, 1>{}); break;
  }
}

template <class T, int V>
void fwd_t(int N, int R, int C, float scale, const void* table, const int* ids, void* out, hipStream_t st) {
  const int x = std::min(64, pow2_at_least((C + V - 1) / V)), y = 256 / x;
  const int blocks = std::min((N + y - 1) / y, 1 << 20);   // beyond 2^20: each several tokens
  hipLaunchKernelGGL((embed_fwd_kernel<T, V>), dim3(blocks), dim3(x, y), 0, st, N, R, C, scale,
                     static_cast<const T*>(table), ids, static_cast<T*>(out));
}

template <class T, int V>
void sum_t(const EmbedPlan& p, float scale, const int* key, const int* ord, const void* g, float* grad,
           hipStream_t st) {
  const int per = 256 / p.group;
  const long long items = (long long)p.chunks * p.slices;
  hipLaunchKernelGGL((embed_sum_kernel<T, V>), dim3((unsigned)((items + per - 1) / per)), dim3(256), 0, st, p.N, p.R,
                     p.C, p.chunk, p.chunks, p.group, p.slices, scale, key, ord, static_cast<const T*>(g), grad, p.part,
                     p.first, p.last);
}

template <int W, int RW, int V>
void join_t(const EmbedPlan& p, float scale, float* grad, hipStream_t st) {
  constexpr int rows = RW == 1 ? 1 : W * RW;
  const int pieces = (p.C + V - 1) / V, group = std::min(64, pow2_at_least(pieces));
  const int y = RW == 1 ? (pieces + 63) / 64 : 1;
  hipLaunchKernelGGL((embed_join_kernel<W, RW, V>), dim3((p.R + rows - 1) / rows, y), dim3(W * 64), 0, st, p.R, p.C,
                     p.chunk, group, scale, p.first, p.last, p.part, grad);
}

}  // namespace

EmbedPlan embed_plan(int N, int R, int C, bool bf16, bool aligned, void* ws) {
  EmbedPlan p{};
  p.N = N, p.R = R, p.C = C;
  int bits = 1;
  while ((1ll << bits) < (long long)R + 1) ++bits;   // keys 0..R
  p.passes = (bits + 7) / 8;
  p.bits = (bits + p.passes - 1) / p.passes;
  p.sort_blocks = (N + kSortItems - 1) / kSortItems;
  p.vec = vec_of(C, bf16, aligned);
  const int pieces = (C + p.vec - 1) / p.vec;
  p.group = std::min(64, pow2_at_least(pieces));
  p.slices = (pieces + p.group - 1) / p.group;
  if (R <= kFewRows) {
    p.windows = (N + kWindow - 1) / kWindow;
    p.part = static_cast<float*>(ws);
    p.bytes = sizeof(float) * (size_t)p.windows * R * C;
    return p;
  }
  // chunks of 32 tokens at least (the partial sums then stay below a
  // sixteenth of what is read), longer once 16 waves per CU have one each
  const long long groups = 256ll * 16 * (64 / p.group);
  const long long want = (long long)N * p.slices / groups;
  p.chunk = (int)std::clamp<long long>((want + 31) / 32 * 32, 32, 512);
  p.chunks = (N + p.chunk - 1) / p.chunk;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t o = at;
    at += (n + 255) / 256 * 256;
    return static_cast<char*>(ws) + o;
  };
  for (int i = 0; i < 2; ++i) {
    p.key[i] = reinterpret_cast<int*>(take(sizeof(int) * (size_t)N));
    p.ord[i] = reinterpret_cast<int*>(take(sizeof(int) * (size_t)N));
  }
  p.hist = reinterpret_cast<int*>(take(sizeof(int) * ((size_t)p.sort_blocks << p.bits)));
  p.total = reinterpret_cast<int*>(take(sizeof(int) * 256));
  p.first = reinterpret_cast<int*>(take(sizeof(int) * (size_t)R));
  p.last = reinterpret_cast<int*>(take(sizeof(int) * (size_t)R));
  p.part = reinterpret_cast<float*>(take(sizeof(float) * (size_t)p.chunks * 2 * C));
  p.bytes = at;
  return p;
}

void launch_embed_fwd(int N, int R, int C, bool is_bf16, bool aligned, float scale, const void* table, const int* ids,
                      void* out, hipStream_t st) {
  dispatch(is_bf16, vec_of(C, is_bf16, aligned), [&](auto t, auto v) {
    fwd_t<decltype(t), decltype(v)::value>(N, R, C, scale, table, ids, out, st);
  });
}

void launch_embed_vjp(const EmbedPlan& p, bool is_bf16, float scale, const int* ids, const void* g, float* grad,
                      hipStream_t st) {
  if (p.windows > 0) {
    const int per = std::max(p.group, 16);   // the threads beyond kWindow / per groups only sort
    dispatch(is_bf16, p.vec, [&](auto t, auto v) {
      using E = decltype(t);
      hipLaunchKernelGGL((embed_window_kernel<E, decltype(v)::value>), dim3(p.windows, p.slices), dim3(kWindow), 0, st,
                         p.N, p.R, p.C, p.group, per, ids, static_cast<const E*>(g), p.part);
    });
    const size_t n = (size_t)p.R * p.C;
    hipLaunchKernelGGL(embed_window_join_kernel, dim3((unsigned)((n + 63) / 64)), dim3(1024), 0, st, p.windows, n, scale,
                       p.part, grad);
    return;
  }
  const int ndig = 1 << p.bits;
  const int* key = ids;
  const int* ord = nullptr;
  const bool small = p.N <= kSmall;
  if (small) {
    hipLaunchKernelGGL(sort_small_kernel, dim3(1 + std::clamp(p.R / (4 * kSmallThreads), 1, 128)), dim3(kSmallThreads), 0,
                       st, p.N, p.R, p.bits, p.passes, ids, p.key[0], p.ord[0], p.first, p.last);
    key = p.key[0];
    ord = p.ord[0];
  }
  for (int s = 0; s < (small ? 0 : p.passes); ++s) {
    int *ko = p.key[s & 1], *oo = p.ord[s & 1];
    hipLaunchKernelGGL(sort_count_kernel, dim3(p.sort_blocks), dim3(kSortThreads), 0, st, p.N, p.R, s * p.bits, ndig,
                       s == 0, key, p.hist);
    hipLaunchKernelGGL(sort_scan_kernel, dim3(ndig), dim3(256), 0, st, p.sort_blocks, p.hist, p.total,
                       s == 0 ? p.R : 0, p.first, p.last);
    hipLaunchKernelGGL(sort_scatter_kernel, dim3(p.sort_blocks), dim3(kSortThreads), 0, st, p.N, p.R, s * p.bits,
                       p.bits, s == 0, key, ord, p.hist, p.total, ko, oo);
    key = ko;
    ord = oo;
  }
  dispatch(is_bf16, p.vec, [&](auto t, auto v) {
    sum_t<decltype(t), decltype(v)::value>(p, scale, key, ord, g, grad, st);
  });
  // few rows, whose runs are long: a block of 16 waves for each and 64
  // channels; many: each wave a run of rows
  if (p.R <= 512)
    join_t<16, 1, 1>(p, scale, grad, st);
  else
    p.vec >= 4 ? join_t<4, 8, 4>(p, scale, grad, st) : join_t<4, 8, 1>(p, scale, grad, st);
}

}  // namespace fc
