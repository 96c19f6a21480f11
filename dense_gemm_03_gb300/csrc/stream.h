// stream.h -- products with few rows or few tiles: as one kernel where a wave of
// clusters covers them, else as fp32 partial sums by K chunks (narrow_stream.cu for halves, i8_stream.cu
// for 8-bit integers) and the kernel that adds them up and finishes the result (stream_sum.cu).
#pragma once

#include <cstddef>
#include <cuda_runtime.h>

#include "internal.h"
#include "lora.h"
#include "row_blocks.h"

namespace gb300 {

// Partial sums: [block of `block` rows][128-column unit][chunk][row of the block][128].
struct StreamParts {
  float* part;
  int chunks, units, block_rows;
  size_t bytes;
  int block;                       // (block_rows: see row_blocks.h)
};
// Chunks per unit (of `kb` steps of 16 KB of W each): see lora_stream.cu.
int plan_chunks(int units, int blocks, int kb, int rows, int sms, int least = 1);

// Longest chunk of K of a folded sum (float results, relu's gradient): the tensor core's
// additions truncate (over 512 products by 0.7e-6 of the sums' norm).
constexpr int kFoldDepth = 512;

// op(X) (M x K, stored K x M where trans_x) times op(W) (K x `cols`; N x K) in halves, or
// X W in 8-bit integers (i8_*); rows on the 16-byte grid.
struct NarrowStream {
  const void *X, *W;
  long long ldx, ldw;
  int K;
  bool trans_x, trans_w;
  bool beside = false;   // see PairDone (internal.h)
};
// Its partial sums; fold: in chunks of kFoldDepth at most.
StreamParts narrow_parts(const NarrowStream& p, int M, int cols, bool fold, const LoraDevice& d);
int narrow_partial(const NarrowStream& p, int M, int cols, bool fold, const StreamParts& parts,
                   const LoraDevice& d, cudaStream_t stream);
StreamParts i8_parts(const NarrowStream& p, int M, int cols, const LoraDevice& d);
int i8_partial(const NarrowStream& p, int M, int cols, const StreamParts& parts,
               const LoraDevice& d, cudaStream_t stream);

// What becomes of the sums S (gate 0: N columns; else 2 N, G and U):
//   gate 0   C := alpha S + beta C (half, or float when f32); with scales S
//            sx[row] sw[column] in the place of S
//   gate 1   C := f(G) .* U, G and U scaled where there are scales
//   gate 2   dG = dC .* U .* f'(G) to C, dU = dC .* f(G) to g.dU
struct StreamSum {
  StreamParts parts;
  void* C;
  long long ldc;
  int M, N;
  float alpha, beta;
  int gate;
  bool f32, scaled;
  bool fold;   // chunks of kFoldDepth at most, as a float result's
  GateArgs g;
};
// The whole product in one launch, finished as `s` says (its parts unused), where one
// wave of clusters covers it.
bool narrow_cluster_suits(const NarrowStream& p, const StreamSum& s, const LoraDevice& d);
int narrow_cluster(const NarrowStream& p, const StreamSum& s, const LoraDevice& d,
                   cudaStream_t stream);
bool i8_cluster_suits(const StreamSum& s, int K, const LoraDevice& d);
int i8_cluster(const NarrowStream& p, const StreamSum& s, const LoraDevice& d,
               cudaStream_t stream);
int stream_sum(const StreamSum& s, const LoraDevice& d, cudaStream_t stream);

}  // namespace gb300
