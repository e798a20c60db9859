// rope_args.h - what the host side of the C ABI and the kernels of fa_rope.cuh share.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace fa {

// The rows of one kind (queries, keys or values) on one side: row of head h and token n of
// batch entry b at data + b * sb + n * sn + h * sh (elements); heads = 0: absent. In a packed
// batch sb is not used and n is the token's index in the tensor.
struct HeadRows {
  __nv_bfloat16* data;
  int heads;
  long long sb, sn, sh;
};

struct RopeArgs {
  HeadRows x[3];      // the projection's rows: queries, keys, values
  HeadRows y[3];      // the attention's rows
  HeadRows g[3];      // backward: the gradients of x (y then holds those of the outputs)
  const float* w[2];  // gains of queries and keys (D values each), or null
  float* dw[2];       // backward: their gradients, or null
  float* partial;     // backward: per-block sums, (blocks, 2, D)
  int norm;
  float eps;
  int rot;                  // rotary_dim: a multiple of 8, at most D; 0 = no rotation
  int axes;
  const float* inv_freq;    // rot / 2
  const uint8_t* pair_axis; // rot / 2, or null (axis 0)
  const int* positions;     // (axes, tokens), or null (the place in the sequence)
  const int* seq_len;       // B real lengths of a padded batch, or null
  const int* cu;            // B + 1 cumulative lengths of a packed batch, or null
  int fill;                 // packed: tokens that no sequence covers are written as zeros
  int B;
  int N;                    // rows per entry; packed: the longest sequence handled
  int tokens;               // B * N, or the packed tensors' tokens
  int splits;               // warps per token
};

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;
// Blocks an SM holds (128 registers per thread); the kernels' grids are persistent. With three or
// four blocks ptxas spills, which costs more than the further warps give (backward on 32 x 2048
// tokens of 3 x 16 heads of 64: 234 us with two blocks, 398 with three).
constexpr int kRopeBlocksPerSm = 2;
// Blocks of the backward at most: its workspace holds the gains' sums of each.
constexpr int kRopeMaxBlocks = 512;

}  // namespace fa
