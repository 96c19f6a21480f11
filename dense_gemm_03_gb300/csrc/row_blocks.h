// row_blocks.h -- how the rows of a streamed product (stream.h) are cut into blocks.
#pragma once

#include <algorithm>

namespace gb300 {

// Rows of a block: all blocks about as long, at most `most`, in 16s; in 64s of an X stored
// transposed with whole 64-row blocks, which one copy then stages (block_of_64s).
inline int block_rows(int M, int most, bool trans_x) {
  const int blocks = (M + most - 1) / most, unit = trans_x && M % 64 == 0 ? 64 : 16;
  return std::min(M, ((M + blocks - 1) / blocks + unit - 1) / unit * unit);
}

// Whether every block of `rows` of the M rows is made of whole 64-row blocks of them.
inline bool block_of_64s(int M, int rows) { return M % 64 == 0 && (rows % 64 == 0 || rows >= M); }

}  // namespace gb300
