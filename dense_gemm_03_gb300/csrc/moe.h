// moe.h -- what the two files of the mixture-of-experts layer share.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

#include "internal.h"
#include "ptx.cuh"

namespace gb300 {

constexpr int kMoeMaxExperts = 1024;
constexpr int kMoeMaxTopk = 32;

struct MoeArgs {
  const uint16_t *X, *Wr, *W1, *W2;
  uint16_t* Y;
  int* ids;
  float* probs;
  int T, H, I, E, topk, renormalize;
  int ldx, ldy;
  float beta;
};

// Whether moe_stream takes the call: weights with 16-byte rows (the TMA rule)
// and X with 16-byte rows.
bool moe_stream_fits(const MoeArgs& m);
// The layer, up to 64 tokens at a time.  Returns a GEMM_* code.
int moe_stream(const MoeArgs& m, int sms, DeviceStatus* st, unsigned long long limit_ns,
               cudaStream_t stream);

__device__ __forceinline__ float moe_h2f(uint16_t b) { return __half2float(__ushort_as_half(b)); }
__device__ __forceinline__ uint16_t moe_f2h(float x) {
  return __half_as_ushort(__float2half_rn(x));
}

// |x| as bits that order like it, or 0 for an infinity or NaN.
__device__ __forceinline__ unsigned int moe_finite_bits(float x) {
  const unsigned int b = __float_as_uint(x) & 0x7FFFFFFFu;
  return b < 0x7F800000u ? b : 0u;
}
// The power of two that brings a magnitude (its bits) into [2^13, 2^14), at most
// 2^126 either way, so that it and its inverse are normal; and that inverse.
__device__ __forceinline__ float moe_scale(unsigned int top) {
  return __int_as_float(min(253, 127 + 13 + 127 - static_cast<int>(top >> 23)) << 23);
}
__device__ __forceinline__ float moe_unscale(float up) {
  return __int_as_float((254 << 23) - __float_as_int(up));
}

// Four entries times `up` as halves, hi and what it leaves out; a hi that is not
// finite stands alone.
__device__ __forceinline__ void moe_split4(float4 v, float up, uint2& hi, uint2& lo) {
  const float x[4] = {up * v.x, up * v.y, up * v.z, up * v.w};
  uint32_t h[2], l[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2 hh = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    const float2 f = __half22float2(hh);
    const __half2 ll = __floats2half2_rn(x[2 * i] - f.x, x[2 * i + 1] - f.y);
    memcpy(h + i, &hh, 4);
    memcpy(l + i, &ll, 4);
    l[i] &= __hlt2_mask(__habs2(hh), __half2half2(__ushort_as_half(0x7C00)));
  }
  hi = make_uint2(h[0], h[1]);
  lo = make_uint2(l[0], l[1]);
}

// The two halves' products with the same weights.  Where those hold an infinity
// the hi part is the result; lo, of either sign or zero, would make it NaN.
__device__ __forceinline__ float moe_join(float hi, float lo) { return isinf(hi) ? hi : hi + lo; }

// Order-preserving key of a float: larger floats have larger keys, -0 and +0
// the same one, NaN the largest.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One warp: the topk largest of logits[0, E) (ties: the lowest index), falling,
// into ids and p[k] = softmax(logits) there, divided by their sum when
// `renormalize`.  The keys stay in registers, NR of 32 per lane (E <= 32 NR).
template <int NR>
__device__ __forceinline__ void select_experts(const float* logits, int E, int topk,
                                               int renormalize, int* ids, float* probs) {
  const int lane = threadIdx.x & 31;
  uint32_t key[NR];
#pragma unroll
  for (int j = 0; j < NR; ++j)   // no logit has key 0
    key[j] = lane + 32 * j < E ? order_key(logits[lane + 32 * j]) : 0u;
  int mine = 0;                  // lane k: the k-th expert
  for (int k = 0; k < topk; ++k) {
    uint32_t best = 0;
#pragma unroll
    for (int j = 0; j < NR; ++j) best = max(best, key[j]);
    const uint32_t most = __reduce_max_sync(0xffffffffu, best);
    uint32_t at = 0xFFFFFFFFu;
#pragma unroll
    for (int j = NR - 1; j >= 0; --j)
      if (key[j] == most) at = static_cast<uint32_t>(lane + 32 * j);
    const uint32_t e = __reduce_min_sync(0xffffffffu, at);
#pragma unroll
    for (int j = 0; j < NR; ++j)
      if (e == static_cast<uint32_t>(lane + 32 * j)) key[j] = 0u;
    if (lane == k) mine = static_cast<int>(e);
  }
  const float top = logits[__shfl_sync(0xffffffffu, mine, 0)];
  float sum = 0.0f;
  for (int e = lane; e < E; e += 32) sum += expf(logits[e] - top);
  float p = lane < topk ? expf(logits[mine] - top) : 0.0f;
  float chosen = p;
  for (int d = 16; d; d >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, d);
    chosen += __shfl_xor_sync(0xffffffffu, chosen, d);
  }
  p /= renormalize ? chosen : sum;
  if (lane < topk) {
    ids[lane] = mine;
    probs[lane] = p;
  }
  __syncwarp();
}

// The same for any E up to the layer's limit.
__device__ __forceinline__ void select_experts(const float* logits, int E, int topk,
                                               int renormalize, int* ids, float* probs) {
  if (E <= 64)
    select_experts<2>(logits, E, topk, renormalize, ids, probs);
  else if (E <= 256)
    select_experts<8>(logits, E, topk, renormalize, ids, probs);
  else
    select_experts<kMoeMaxExperts / 32>(logits, E, topk, renormalize, ids, probs);
}

}  // namespace gb300
