// gb_layers.h — what the C-ABI layer of the token-sum layers
// (gb_layers_api.cpp) and their kernels (gb_norm.hip, gb_embed.hip) share.
// Not installed; the public ABI is include/gbreduce.h.
//
// Every launcher assumes arguments that gb_layers_api.cpp validated, and
// returns hipSuccess or the launch error.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "gbreduce.h"

namespace gb {

// A 2-D array of unit stride along its rows; stride in elements.
struct Rows {
  void* p;
  size_t stride;
};

// ---------------------------------------------------------------------------
// Layer norm
// ---------------------------------------------------------------------------
struct NormArgs {
  Rows y, x;
  size_t rows;
  uint32_t cols;
  int dtype;        // of x and y
  int param_dtype;  // of w and b
  const void* w;    // NULL: ones
  const void* b;    // NULL: zeros
  float eps;
  float* mean;  // NULL: not stored
  float* rstd;
};
hipError_t launch_layer_norm(const NormArgs& a, hipStream_t stream);

struct NormGradArgs {
  Rows dx, dy, x;  // dx.p NULL: not computed
  size_t rows;
  uint32_t cols;
  int dtype, param_dtype, grad_dtype;
  const float* mean;
  const float* rstd;
  const void* w;  // NULL: ones
  void* dw;       // NULL: not computed
  void* db;
  bool accumulate;
  float* partials;  // float[2 * groups][partial_stride]
  size_t partial_stride;
};
// Workgroups of the backward pass, each of which leaves one row of partial
// sums for dw and one for db.
uint32_t norm_grad_groups(size_t rows, size_t cols, int dtype);
inline size_t norm_partial_stride(size_t cols) { return (cols + 3) / 4 * 4; }
hipError_t launch_layer_norm_grad(const NormGradArgs& a, hipStream_t stream);

// ---------------------------------------------------------------------------
// Embedding
// ---------------------------------------------------------------------------
struct LookArgs {
  Rows out, table;
  const void* ids;
  size_t tokens, vocab, dim;
  int64_t first;
  float scale;
  int out_dtype, table_dtype, id_dtype;
};
hipError_t launch_embedding(const LookArgs& a, hipStream_t stream);

// Occurrences of an id that are added one after the other before their sums
// are added in turn: the unit of the sum's order that the ABI documents.
constexpr uint32_t kFold = 64;

// A run of more than one fold in the join's work list.
constexpr size_t kLongRunBytes = 12;

// Tokens that one workgroup sorts alone; more take a launch pair per digit.
constexpr uint32_t kSortSmall = 8192;
constexpr uint32_t kSortThreads = 1024;
constexpr uint32_t kSortTile = 2048;    // tokens that a workgroup of the digit passes ranks at a time
constexpr uint32_t kSortBlocks = 128;   // workgroups of a digit pass, at most
constexpr uint32_t kSortDigitBits = 10; // bins of a digit: one per lane of a workgroup, at most
constexpr uint32_t kSortLeastBits = 8;  // and at least 256, or few lanes add up many lanes' counts

// Byte offsets in the workspace of the embedding's backward pass.
struct LookGradLayout {
  size_t count;       // uint32[2]: tokens that name a row, and runs of more than one fold
  size_t keys[2];     // uint32[tokens]: row of a token, and
  size_t tokens[2];   // uint32[tokens]: its number; two of each, a digit pass reads one and writes the other
  size_t hist;        // uint32[workgroups][bins] of a digit pass
  size_t named;       // uint8[vocab]: whether a token names the row
  size_t long_runs;   // kLongRunBytes[tokens / (kFold + 1)]: the runs of more than one fold
  size_t partials;    // float[2 * windows][stride]
  size_t total;
};
inline size_t look_windows(size_t tokens) { return (tokens + kFold - 1) / kFold; }
inline size_t look_partial_stride(size_t dim) { return (dim + 3) / 4 * 4; }
inline uint32_t sort_blocks(size_t tokens) {
  const size_t tiles = (tokens + kSortTile - 1) / kSortTile;
  return (uint32_t)(tiles < kSortBlocks ? tiles : kSortBlocks);
}
inline LookGradLayout look_grad_layout(size_t tokens, size_t vocab, size_t dim) {
  const auto up = [](size_t b) { return (b + 255) / 256 * 256; };
  const bool digits = tokens > kSortSmall;
  LookGradLayout l;
  size_t at = 0;
  l.count = at, at += 256;
  for (int i = 0; i < 2; i++) {
    l.keys[i] = at, at += i == 0 || digits ? up(4 * tokens) : 0;
    l.tokens[i] = at, at += i == 0 || digits ? up(4 * tokens) : 0;
  }
  l.hist = at, at += digits ? up((size_t)sort_blocks(tokens) * 4 << kSortDigitBits) : 0;
  l.named = at, at += up(vocab);
  l.long_runs = at, at += up(kLongRunBytes * (tokens / (kFold + 1)));
  l.partials = at, at += tokens > kFold ? up(2 * look_windows(tokens) * look_partial_stride(dim) * 4) : 0;
  l.total = at;
  return l;
}

struct LookGradArgs {
  Rows dtable, dout;
  const void* ids;
  size_t tokens, vocab, dim;
  int64_t first, padding;
  float scale;
  int dtype, grad_dtype, id_dtype;  // of dout, dtable and ids
  bool accumulate;
  char* workspace;
};
hipError_t launch_embedding_grad(const LookGradArgs& a, hipStream_t stream);

// The workgroups of the table's sums: [0, sums) add tokens, [sums, sums +
// zeros) clear rows without one.  A launch takes those from base on, at most
// kSumLaunch of them: a launch of 2^32 lanes would be refused, and 2^30 rows
// of few columns, or 2^30 tokens, come to more.
struct SumGrid {
  size_t units;          // windows times slabs, a wavefront each
  uint32_t slabs;        // of a row
  uint32_t sums, zeros;  // multiples of the XCDs, as is base
  uint32_t zero_each;    // rows a workgroup looks after
  uint32_t base;
};
constexpr uint32_t kSumLaunch = 1u << 23;

}  // namespace gb
