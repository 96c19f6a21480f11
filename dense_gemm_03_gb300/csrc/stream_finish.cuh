// stream_finish.cuh -- what becomes of VEC neighbouring sums of a row (StreamSum).
#pragma once
#include "gate.cuh"
#include "stream.h"

namespace gb300 {
namespace {

template <int VEC>
__device__ __forceinline__ void load_half(const uint16_t* p, bool vec, int n, float (&v)[VEC]) {
  if (VEC == 4 && vec) {
    const uint2 q = *reinterpret_cast<const uint2*>(p);
    const float2 a = lora_h2f2(q.x), b = lora_h2f2(q.y);
    v[0] = a.x; v[VEC > 1 ? 1 : 0] = a.y; v[VEC > 2 ? 2 : 0] = b.x; v[VEC > 3 ? 3 : 0] = b.y;
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = i < n ? lora_h2f(p[i]) : 0.0f;
  }
}

template <int VEC>
__device__ __forceinline__ void store_half(uint16_t* p, bool vec, int n, const float (&v)[VEC]) {
  if (VEC == 4 && vec) {
    uint2 q;
    q.x = lora_f2h(v[0]) | static_cast<uint32_t>(lora_f2h(v[VEC > 1 ? 1 : 0])) << 16;
    q.y = lora_f2h(v[VEC > 2 ? 2 : 0]) | static_cast<uint32_t>(lora_f2h(v[VEC > 3 ? 3 : 0])) << 16;
    *reinterpret_cast<uint2*>(p) = q;
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (i < n) p[i] = lora_f2h(v[i]);
  }
}

// Columns c .. c + n - 1 of `row`: s (and U's sums u, behind a gate) finished and
// stored; v: n == VEC and the rows of the results, and dC's, are on the grid of VEC
// elements.
template <int GATE, bool F32, bool SCALED, int VEC>
__device__ __forceinline__ void stream_finish(const StreamSum& p, int row, int c, int n, bool v,
                                              float (&s)[VEC], float (&u)[VEC]) {
  const long long at = row * p.ldc + c;
  if constexpr (SCALED) {
    const float sx = p.g.sx ? __ldg(p.g.sx + row) : 1.0f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      s[i] = s[i] * sx * (p.g.sw && i < n ? __ldg(p.g.sw + c + i) : 1.0f);
      if constexpr (GATE != 0) u[i] = u[i] * sx * (p.g.sw && i < n ? __ldg(p.g.sw + p.N + c + i) : 1.0f);
    }
  }
  if constexpr (GATE == 0) {
    if constexpr (F32) {
      float* const dst = static_cast<float*>(p.C) + at;
      if (VEC == 4 && v) {
        float4 old = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (p.beta != 0.0f) old = *reinterpret_cast<const float4*>(dst);
        const float o[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          s[i] = p.beta != 0.0f ? fmaf(p.alpha, s[i], p.beta * o[i]) : p.alpha * s[i];
        *reinterpret_cast<float4*>(dst) = make_float4(s[0], s[VEC > 1 ? 1 : 0], s[VEC > 2 ? 2 : 0],
                                                      s[VEC > 3 ? 3 : 0]);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          if (i < n) dst[i] = p.beta != 0.0f ? fmaf(p.alpha, s[i], p.beta * dst[i]) : p.alpha * s[i];
      }
    } else {
      uint16_t* const dst = static_cast<uint16_t*>(p.C) + at;
      float old[VEC];
      if (p.beta != 0.0f) load_half<VEC>(dst, v, n, old);
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        s[i] = p.beta != 0.0f ? fmaf(p.alpha, s[i], p.beta * old[i]) : p.alpha * s[i];
      store_half<VEC>(dst, v, n, s);
    }
  } else if constexpr (GATE == 1) {
    gate_dispatch(p.g.act, [&](auto act) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) s[i] = gate_value<decltype(act)::value>(s[i]) * u[i];
    });
    store_half<VEC>(static_cast<uint16_t*>(p.C) + at, v, n, s);
  } else {
    float dc[VEC];
    load_half<VEC>(p.g.dC + row * p.g.lddc + c, v, n, dc);
    gate_dispatch(p.g.act, [&](auto act) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        float df;
        const float f = gate_both<decltype(act)::value>(s[i], df);
        s[i] = dc[i] * u[i] * df;
        u[i] = dc[i] * f;
      }
    });
    store_half<VEC>(static_cast<uint16_t*>(p.C) + at, v, n, s);
    store_half<VEC>(p.g.dU + at, v, n, u);
  }
}

}  // namespace
}  // namespace gb300
