// Scaled lookup of table rows and its gradient (launch interface).
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>

namespace fc {

// Workspace of the gradient: sums of a few rows per window of tokens, or sorted
// keys and order (two buffers each), digit counts, run bounds per row, partial
// sums of runs cut by a chunk edge.
struct EmbedPlan {
  int N, R, C;
  int windows;           // of tokens, for tables of few rows; else 0
  int passes, bits;      // radix sort: digits of `bits` bits
  int sort_blocks;       // blocks of the sort's passes
  int chunk, chunks;     // sorted tokens per chunk of the sum, number of chunks
  int group, slices;     // lanes that share a row, channel slices of a row
  int vec;               // channels per lane
  size_t bytes;
  int *key[2], *ord[2], *hist, *total, *first, *last;
  float* part;
};
EmbedPlan embed_plan(int N, int R, int C, bool bf16, bool aligned, void* ws);

void launch_embed_fwd(int N, int R, int C, bool bf16, bool aligned, float scale, const void* table, const int* ids,
                      void* out, hipStream_t st);
void launch_embed_vjp(const EmbedPlan& p, bool bf16, float scale, const int* ids, const void* g, float* grad,
                      hipStream_t st);

}  // namespace fc
