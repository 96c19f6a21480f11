// operands.h -- operands of the calls made of several kernels: alignment checks
// and copies onto the 16-byte grid.
#pragma once

#include <algorithm>
#include <initializer_list>

#include "lora.h"

namespace gb300 {

// Largest size of the calls below: sizes are rounded up to tiles in 32 bits.
constexpr int kMaxDim = 0x7fffffff - 1023;

inline bool misaligned(std::initializer_list<const void*> ptrs, size_t elem) {
  uintptr_t bits = 0;
  for (const void* p : ptrs) bits |= reinterpret_cast<uintptr_t>(p);
  return (bits & (elem - 1)) != 0;
}

// An operand that TMA cannot read where it lies (rows off the 16-byte grid) is
// copied into rows that are on it, zero-padded to a multiple of eight columns;
// `pad` asks for the copy whenever the width itself is no such multiple.
struct Aligned {
  const uint16_t* src;
  int ld;
  long long rows;
  int cols;
  bool copy;
  Aligned(const uint16_t* p, int ld_, long long rows_, int cols_, bool wanted, bool pad = false)
      : src(p), ld(ld_), rows(rows_), cols(cols_) {
    copy = wanted && ((reinterpret_cast<uintptr_t>(p) & 15u) != 0 || ld % 8 != 0 ||
                      (pad && cols % 8 != 0));
  }
  int ld_copy() const { return (cols + 7) / 8 * 8; }
  size_t bytes() const {
    return copy ? lora_round256(2 * static_cast<size_t>(rows) * ld_copy()) : 0;
  }
};

// Makes the copies that are needed, in `buf`, and points *ptr and *ld at them.
struct Operand {
  Aligned a;
  const uint16_t** ptr;
  int* ld;
};

inline int align_operands(std::initializer_list<Operand> ops, uint8_t* buf, int sms, cudaStream_t stream,
                          bool early = false) {
  RealignBatch batch{};
  auto flush = [&]() {
    if (batch.n == 0) return GEMM_OK;
    batch.early = early;
    const cudaError_t e = launch_realign_f16(batch, stream);
    batch = RealignBatch{};
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
  };
  for (const Operand& o : ops) {
    if (!o.a.copy) continue;
    if (o.a.rows > 0x7fffffffll) return GEMM_ERR_ARG;
    uint16_t* const dst = reinterpret_cast<uint16_t*>(buf);
    buf += o.a.bytes();
    const int ld2 = o.a.ld_copy();
    const long long blocks = (o.a.rows * (ld2 / 8) + 255) / 256;
    batch.job[batch.n] = RealignJob{o.a.src, o.a.ld, dst, ld2, static_cast<int>(o.a.rows), o.a.cols};
    batch.end[batch.n] = (batch.n ? batch.end[batch.n - 1] : 0) +
                         static_cast<int>(std::max(1ll, std::min(blocks, 8ll * sms)));
    *o.ptr = dst;
    *o.ld = ld2;
    if (++batch.n == 3)
      if (int rc = flush()) return rc;
  }
  return flush();
}

}  // namespace gb300
