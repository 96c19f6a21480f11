// i8_convert.cuh -- 8-bit integers as halves, exactly.
//
//   byte b = q + 128 (q xor 0x80)  ->  half 0x6400 | b = 1024 + b  ->  minus 1152 = q
// two byte permutes and two packed subtractions for four integers.
#pragma once
#include <cstdint>
#include <cstring>
#include <cuda_fp16.h>

namespace gb300 {

// Four 8-bit integers as halves.
__device__ __forceinline__ uint2 i8_halves(uint32_t w) {
  const uint32_t b = w ^ 0x80808080u;
  const uint32_t lo = __byte_perm(b, 0x64646464u, 0x4140), hi = __byte_perm(b, 0x64646464u, 0x4342);
  const __half2 off = __half2half2(__ushort_as_half(0x6480));
  __half2 l, h;
  memcpy(&l, &lo, 4);
  memcpy(&h, &hi, 4);
  l = __hsub2(l, off);
  h = __hsub2(h, off);
  uint2 r;
  memcpy(&r.x, &l, 4);
  memcpy(&r.y, &h, 4);
  return r;
}

// 16 of them, as two 16-byte pieces.
__device__ __forceinline__ void i8_halves16(uint4 q, uint4& first, uint4& second) {
  const uint2 a = i8_halves(q.x), b = i8_halves(q.y), c = i8_halves(q.z), d = i8_halves(q.w);
  first = make_uint4(a.x, a.y, b.x, b.y);
  second = make_uint4(c.x, c.y, d.x, d.y);
}

}  // namespace gb300
