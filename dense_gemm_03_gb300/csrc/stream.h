// stream.h -- products with few rows or few tiles as fp32 partial sums by K chunks
// (row_stream in lora_stream.cu for halves, i8_stream.cu for 8-bit integers) and
// the kernel that adds them up and finishes the result (stream_sum.cu).
#pragma once

#include <cstddef>
#include <cuda_runtime.h>

#include "internal.h"
#include "lora.h"

namespace gb300 {

// Partial sums: [block of `block` rows][128-column unit][chunk][row of the block][128].
struct StreamParts {
  float* part;
  int chunks, units, block_rows;   // block_rows = min(M, block)
  size_t bytes;
  int block;
};
// Chunks per unit (of `kb` steps of 16 KB of W each): see lora_stream.cu.
int plan_chunks(int units, int blocks, int kb, int rows, int sms, int least = 1);

// X (M x K, or K x M) times W (K x N, or N x K), rows on the 16-byte grid.
struct RowStream {
  const uint16_t *X, *W;
  long long ldx, ldw;
  int M, N, K;
  bool trans_x, trans_w;
  bool fold;   // chunks of at most kFoldDepth, for a float result
};
constexpr int kFoldDepth = 2048;
StreamParts row_stream_parts(const RowStream& p, int sms);   // with part == nullptr
int row_stream(const RowStream& p, const StreamParts& parts, const LoraDevice& d,
               cudaStream_t stream);

// X (M x K) times W (K x N) in 8-bit integers, rows on the 16-byte grid.
struct I8Stream {
  const int8_t *X, *W;
  long long ldx, ldw;
  int M, N, K;
};
StreamParts i8_stream_parts(const I8Stream& p, int sms);
int i8_stream(const I8Stream& p, const StreamParts& parts, const LoraDevice& d, bool early,
              cudaStream_t stream);

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
  GateArgs g;
};
int stream_sum(const StreamSum& s, const LoraDevice& d, cudaStream_t stream);

}  // namespace gb300
