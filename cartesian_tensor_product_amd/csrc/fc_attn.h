// Attention among the rows of each segment (launch interface).
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

namespace fc {

inline constexpr int kAttnMaxDim = 128;
inline constexpr int kAttnMaxHeads = 256;

struct AttnArgs {
  int nq, nk, S, hq, hk, G, D;   // G = hq / hk query heads share a key head
  int64_t qs, ks, vs;            // row strides (elements)
  float scale, cap;              // cap 0: none
  bool causal;
  const int *seg_q, *seg_k, *prefix;
  const void *q, *k, *v;
  const float *slope, *pos_q, *pos_k;   // all null without the distance bias
  // forward outputs, inputs of the VJP
  void* out;
  float* lse;
  // VJP
  const void* g;
  void *gq, *gk, *gv;
  float *g_slope, *g_pos_q, *g_pos_k;
  bool self_pos;                 // pos_k is pos_q: g_pos_q takes both parts
};

// Workspace of one call.  op 0: forward, 1: VJP.
size_t attn_workspace_bytes(const AttnArgs& a, bool bf16, int op);
void launch_attn_fwd(const AttnArgs& a, bool bf16, void* ws, hipStream_t st);
void launch_attn_vjp(const AttnArgs& a, bool bf16, void* ws, hipStream_t st);

// ------------------------------------------------- between the units --

// Partial results when the walked axis is split, and what passes between
// the kernels of the VJP.
struct AttnPart {
  int splits;
  float* o;       // fwd: [splits][nq hq][D], normalised per split; VJP: partial gradients
  float* o2;      // VJP over keys: partial value gradients [splits][nk hk][D]
  float* lse;     // fwd: [splits][nq hq]
  float* delta;   // VJP: [dsplits][nq hq]
  int dsplits;    // 1 unless the delta pass is split
  bool exact;     // delta comes from the delta pass, else the query pass forms <g, out>
  float* row;     // VJP: [splits][nq hq][4] position and slope gradients of a query row, or null
  float* col;     // VJP: [splits][nk hk][4] position gradients of a key row, or null
};

enum AttnPass { kAttnFwd, kAttnDelta, kAttnQuery, kAttnKey };
enum AttnMode { kOne, kCols, kRows };   // how the waves of a block share its work
struct AttnLaunch {
  AttnPass pass;
  AttnMode mode;
  int hb;         // key heads per wave, 1 or (forward with a bias) 2
};

// Whether the forward may hold two key heads per wave (they share the
// distances): their columns, accumulators and row tiles have to fit, and fp32
// rows have three parts.  In the VJP one head per wave was as fast or faster
// at every size (more waves fit).
constexpr bool attn_two_heads(bool bf16, int DP) { return DP <= (bf16 ? 64 : 32); }
// Row tiles too large for a wave alone: kCols is the only mode.
constexpr bool attn_cols_only(bool bf16, int DP) { return !bf16 && DP > 64; }

// One function per element type and padded head dimension (own units).
template <class T, int DP>
void attn_launch(const AttnLaunch& l, const AttnArgs& a, const AttnPart& p, hipStream_t st);

}  // namespace fc
