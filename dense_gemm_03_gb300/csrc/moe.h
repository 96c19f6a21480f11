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

// Order-preserving key of a float: larger floats have larger keys, -0 and +0
// the same one, NaN the largest.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One warp: the topk largest of logits[0, E) (ties: the lowest index), falling,
// into ids and p[k] = softmax(logits) there, divided by their sum when
// `renormalize`.  `taken` holds E marks.
__device__ __forceinline__ void select_experts(const float* logits, uint8_t* taken, int E, int topk,
                                               int renormalize, int* ids, float* probs) {
  const int lane = threadIdx.x & 31;
  float sum = 0.0f, top = 0.0f, chosen = 0.0f;
  for (int e = lane; e < E; e += 32) taken[e] = 0;
  __syncwarp();
  for (int k = 0; k < topk; ++k) {
    uint32_t best = 0;
    int arg = E;
    for (int e = lane; e < E; e += 32)
      if (!taken[e]) {
        const uint32_t key = order_key(logits[e]);
        if (arg == E || key > best) {
          best = key;
          arg = e;
        }
      }
    const uint32_t most = __reduce_max_sync(0xffffffffu, arg < E ? best : 0u);
    const uint32_t first =
        __reduce_min_sync(0xffffffffu, (arg < E && best == most) ? static_cast<uint32_t>(arg)
                                                                 : 0xFFFFFFFFu);
    const int e = static_cast<int>(first);
    if (k == 0) {
      top = logits[e];
      for (int j = lane; j < E; j += 32) sum += expf(logits[j] - top);
      for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    }
    const float p = expf(logits[e] - top) / sum;
    chosen += p;
    if (lane == 0) {
      taken[e] = 1;
      ids[k] = e;
      probs[k] = p;
    }
    __syncwarp();
  }
  if (renormalize)
    for (int k = lane; k < topk; k += 32) probs[k] = probs[k] / chosen;
  __syncwarp();
}

}  // namespace gb300
