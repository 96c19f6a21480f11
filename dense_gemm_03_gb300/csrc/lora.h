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

// The forward for a few rows (M <= kLoraStreamRows): W streamed once.  Every
// operand has rows on the 16-byte grid; A has zero columns up to a multiple of
// eight.
constexpr int kLoraStreamRows = 128;
size_t lora_stream_bytes(const LoraArgs& p, int sms);
int lora_stream(const LoraArgs& p, uint16_t* C, int ldc, float alpha, float beta, void* scratch,
                const LoraDevice& d, cudaStream_t stream);

// The low-rank products of many rows (lora_shrink.cu): V = s x F[a], F[a] a
// C x R matrix, or R x C when k_major.
struct LoraShrinkJob {
  const uint16_t* x;
  long long ldx;
  int C;                  // columns of x
  const uint16_t* F;
  long long ldf, f_stride;
  int k_major;
  float* V;               // out: [M][ldv]
  int tiles;
};
struct LoraShrinkPlan {
  LoraShrinkJob job[2];
  int njobs;
  const int* ids;
  const float* scales;
  int M, R, adapters;
  int ldv;                // R rounded up to 4
  // weights to mark adapters by (NULL: neither marks nor lists are wanted)
  const uint16_t* check;
  long long ld_check, check_stride;
  int check_rows, check_cols;
  int *lists, *bad;       // out: LoraTailArgs::lists and bad
};
size_t lora_shrink_bytes(const LoraShrinkPlan& p, int sms);
// `counters`: 8 words per 128 rows, zero before and after.
int lora_shrink(LoraShrinkPlan& p, void* scratch, unsigned int* counters, const LoraDevice& d,
                cudaStream_t stream);

// The adapters' gradients (lora_outer.cu): dA from X and U, dB from V and G;
// either may be NULL.
struct LoraOuter {
  const uint16_t *X, *G;
  long long ldx, ldg;
  const float *U, *V;     // [M][ldv]
  int ldv;
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

inline size_t lora_round256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace gb300
