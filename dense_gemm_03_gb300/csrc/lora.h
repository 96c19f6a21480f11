// lora.h -- what the files of the adapter products share.
#pragma once

#include <algorithm>
#include <cstdint>
#include <cuda_fp16.h>

#include "gemm.h"
#include "internal.h"
#include "ptx.cuh"

namespace gb300 {

constexpr int kLoraMaxRank = 128;

struct LoraArgs {
  const uint16_t *X, *W, *A, *B;
  const int* ids;
  const float* scales;
  int M, N, K, R, adapters;
  int ldx, ldw, lda, ldb;
  long long a_stride() const { return static_cast<long long>(K) * lda; }
  long long b_stride() const { return static_cast<long long>(R) * ldb; }
};

// What a launch needs to know of the device.
struct LoraDevice {
  int sms;
  DeviceStatus* status;
  unsigned long long wait_limit_ns;
};

// C := alpha (X W + V F[a]) + beta C by K chunks with their sum in a kernel of
// its own (lora_stream.cu): F[a] is R x N, or N x R when trans, and W then N x K.
// V is given ([M][ldv]), or made here from A (lora_stream_shrinks; A then has
// zero columns up to a multiple of eight).  Operands have rows on the 16-byte
// grid, except C.
struct LoraStream {
  const uint16_t *X, *W;
  uint16_t* C;
  long long ldx, ldw, ldc;
  int M, N, K, R, adapters, trans;
  const uint16_t* F;
  long long ldf, f_stride;
  const float* V;
  int ldv;
  const uint16_t* A;
  long long lda, a_stride;
  const int* ids;
  const float* scales;
  float alpha, beta;
};
// Whether the chunks suit an M x N result better than whole 256 x 256 tiles on
// CTA pairs: a few rows, or so few tiles that half the pairs would be idle.
bool lora_stream_suits(int M, int N, int sms);
// Whether it makes V itself better than lora_shrink does.
bool lora_stream_shrinks(int M, int K, int R);
size_t lora_stream_bytes(const LoraStream& p, int sms);
int lora_stream(const LoraStream& p, void* scratch, const LoraDevice& d, cudaStream_t stream);

// The low-rank products of many rows (lora_shrink.cu): V = s x F[a], F[a] a
// C x R matrix, or R x C when k_major.
struct LoraShrinkJob {
  const uint16_t* x;
  long long ldx;
  int C;                  // columns of x
  const uint16_t* F;
  long long ldf, f_stride;
  int k_major;
  int want;               // kLoraPacked, kLoraScaled
  float* V;               // out: [M][ldv]
  // out: V as hi and lo halves, [M][chunk of 32 ranks][32 hi, 32 lo]; scaled by
  // a power of two for each adapter of 128 rows, whose inverses are unscale[M]
  uint16_t *packed, *scaled;
  uint8_t* apart;         // beside packed: LoraTailArgs::apart
  float* unscale;
  int tiles;
};
constexpr int kLoraPacked = 1, kLoraScaled = 2;
struct LoraShrinkPlan {
  LoraShrinkJob job[2];
  int njobs;
  int max_c;              // of all the jobs that the operator can have
  long long sum_c;
  const int* ids;
  const float* scales;
  int M, R, adapters;
  int ldv;                // R rounded up to 4
  // weights to mark adapters by (NULL: neither marks nor lists are wanted)
  const uint16_t* check;
  long long ld_check, check_stride;
  int check_rows, check_cols;
  float large;            // magnitude past which a weight counts as large
  int *lists, *bad;       // out: LoraTailArgs::lists and bad
};
size_t lora_shrink_bytes(const LoraShrinkPlan& p);
int lora_shrink(LoraShrinkPlan& p, void* scratch, const LoraDevice& d, cudaStream_t stream);

// The same row by row (lora_rows.cu), without lists and marks.  F's rows along K
// (not k_major) have zero columns up to a multiple of eight.
bool lora_rows_suit(const LoraShrinkPlan& p);
size_t lora_rows_bytes(const LoraShrinkPlan& p, int sms);
int lora_rows(LoraShrinkPlan& p, void* scratch, const LoraDevice& d, cudaStream_t stream);
// Its first kernel: V as [row][slice][R], R a multiple of eight.
constexpr int kLoraRowSlices = 16;
struct LoraRowsJob {
  const uint16_t* x;
  long long ldx;
  int C;
  const uint16_t* F;
  long long ldf, f_stride;
  int k_major;
  float* V;
  int ranks;              // of F; V's other columns are zero
};
struct LoraRows {
  LoraRowsJob job[2];
  int njobs, slices;
  const int* ids;
  const float* scales;
  int M, R, adapters;
};
cudaError_t launch_lora_rows(const LoraRows& p, cudaStream_t stream);

// The adapters' gradients (lora_outer.cu): dA from X and U, dB from V and G;
// either may be NULL.
struct LoraOuter {
  const uint16_t *X, *G;
  long long ldx, ldg;
  const LoraShrinkJob *U, *V;   // their scaled halves
  const int* ids;
  float *dA, *dB;
  int M, N, K, R, adapters;
  float alpha, beta;
};
constexpr int kLoraMaxAdapters = 16384;   // of a gradient (its table of places)
size_t lora_outer_bytes(const LoraOuter& o);
int lora_outer(const LoraOuter& o, void* scratch, const LoraDevice& d, cudaStream_t stream);

__device__ __forceinline__ float lora_h2f(uint16_t b) { return __half2float(__ushort_as_half(b)); }
__device__ __forceinline__ uint16_t lora_f2h(float x) {
  return __half_as_ushort(__float2half_rn(x));
}
__device__ __forceinline__ float2 lora_h2f2(uint32_t bits) {
  __half2 h;
  memcpy(&h, &bits, 4);
  return __half22float2(h);
}

// Four entries as hi halves at o and lo halves 32 further; past the half range
// hi is infinite and stands alone.
__device__ __forceinline__ void lora_store_split(uint16_t* o, float4 v) {
  const __half2 h0 = __floats2half2_rn(v.x, v.y), h1 = __floats2half2_rn(v.z, v.w);
  const float2 f0 = __half22float2(h0), f1 = __half22float2(h1);
  const __half2 l0 = __floats2half2_rn(isinf(f0.x) ? 0.0f : v.x - f0.x, isinf(f0.y) ? 0.0f : v.y - f0.y);
  const __half2 l1 = __floats2half2_rn(isinf(f1.x) ? 0.0f : v.z - f1.x, isinf(f1.y) ? 0.0f : v.w - f1.y);
  uint32_t b[4];
  memcpy(b, &h0, 4);
  memcpy(b + 1, &h1, 4);
  memcpy(b + 2, &l0, 4);
  memcpy(b + 3, &l1, 4);
  *reinterpret_cast<uint2*>(o) = make_uint2(b[0], b[1]);
  *reinterpret_cast<uint2*>(o + 32) = make_uint2(b[2], b[3]);
}

// The two halves' products with the same factors.  Where those hold an infinity
// the hi part is the result; lo, of either sign or zero, would make it NaN.
__device__ __forceinline__ float lora_join(float hi, float lo) { return isinf(hi) ? hi : hi + lo; }

// The power of two that brings a largest finite magnitude `top` into [2^13,
// 2^14): its exponent, at most 126 either way, so that it and its inverse are
// normal (below 2^-112 the largest scaled magnitude is less, and has bits enough).
__device__ __forceinline__ int lora_scale_exponent(float top) {
  return top > 0.0f ? max(-126, min(126, 13 - ilogbf(top))) : 0;
}
__device__ __forceinline__ float lora_power(int e) { return __int_as_float((127 + e) << 23); }
// The largest finite magnitude of four, as bits that order like it.
__device__ __forceinline__ unsigned int lora_top_bits(float4 v) {
  const float m[4] = {fabsf(v.x), fabsf(v.y), fabsf(v.z), fabsf(v.w)};
  float top = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (m[j] < __int_as_float(0x7F800000)) top = fmaxf(top, m[j]);
  return __float_as_uint(top);
}

inline size_t lora_round256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace gb300
