// moe.cu -- a whole mixture-of-experts layer: argument checks, path choice and
// the CUDA-core kernels.
//
//   l = x Wr; the topk experts of largest l, ties to the lowest index;
//   p_k = exp(l_k - max l) / sum over all experts (or over the chosen ones);
//   y = sum_k p_k (silu(x W1g[e_k]) .* (x W1u[e_k])) W2[e_k] + beta y
//
// The three kernels of this file (route, up, down) serve every alignment: one
// block per token, then per (token, choice, 64 columns), then per (token, 64
// columns); all sums fp32, the gated product kept in fp32.
#include <cuda_fp16.h>

#include <algorithm>
#include <cstdint>
#include <initializer_list>

#include "gemm.h"
#include "moe.h"

namespace gb300 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxExperts = kMoeMaxExperts;
constexpr int kMaxTopk = kMoeMaxTopk;

__device__ __forceinline__ float h2f(uint16_t b) { return moe_h2f(b); }
__device__ __forceinline__ uint16_t f2h(float x) { return moe_f2h(x); }

__global__ void __launch_bounds__(kThreads)
    moe_route_kernel(const uint16_t* __restrict__ X, long long ldx, const uint16_t* __restrict__ Wr,
                     int T, int H, int E, int topk, int renormalize, int* __restrict__ ids,
                     float* __restrict__ probs, int* __restrict__ ids_out,
                     float* __restrict__ probs_out) {
  __shared__ float logits[kMaxExperts];
  __shared__ float part[kWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int t = blockIdx.x; t < T; t += gridDim.x) {
    const uint16_t* x = X + static_cast<long long>(t) * ldx;
    for (int e0 = 0; e0 < E; e0 += 32) {
      float s = 0.0f;
      if (e0 + lane < E)
        for (int h = warp; h < H; h += kWarps)
          s = fmaf(h2f(x[h]), h2f(Wr[static_cast<long long>(h) * E + e0 + lane]), s);
      part[warp][lane] = s;
      __syncthreads();
      if (warp == 0 && e0 + lane < E) {
        float l = 0.0f;
        for (int w = 0; w < kWarps; ++w) l += part[w][lane];
        logits[e0 + lane] = l;
      }
      __syncthreads();
    }
    if (warp == 0) {
      int* const id = ids + static_cast<long long>(t) * topk;
      float* const p = probs + static_cast<long long>(t) * topk;
      select_experts(logits, E, topk, renormalize, id, p);
      for (int k = lane; k < topk; k += 32) {
        if (ids_out) ids_out[static_cast<long long>(t) * topk + k] = id[k];
        if (probs_out) probs_out[static_cast<long long>(t) * topk + k] = p[k];
      }
    }
    __syncthreads();
  }
}

// hid[t, k][j] = silu(x W1g[e]) * (x W1u[e]) at 64 columns j; four threads
// share a column's sum.
__global__ void __launch_bounds__(kThreads)
    moe_up_kernel(const uint16_t* __restrict__ X, long long ldx, const uint16_t* __restrict__ W1,
                  const int* __restrict__ ids, float* __restrict__ hid, int T, int H, int I,
                  int topk) {
  __shared__ float sg[4][64], su[4][64];
  const int tiles = (I + 63) / 64;
  const long long items = static_cast<long long>(T) * topk * tiles;
  const int c = threadIdx.x & 63, q = threadIdx.x >> 6;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const long long pair = it / tiles;
    const int j = static_cast<int>(it % tiles) * 64 + c;
    const uint16_t* x = X + pair / topk * ldx;
    const uint16_t* w = W1 + static_cast<long long>(ids[pair]) * H * (2ll * I);
    float g = 0.0f, u = 0.0f;
    if (j < I)
      for (int h = q; h < H; h += 4) {
        const float xv = h2f(x[h]);
        const uint16_t* r = w + static_cast<long long>(h) * (2ll * I) + j;
        g = fmaf(xv, h2f(r[0]), g);
        u = fmaf(xv, h2f(r[I]), u);
      }
    sg[q][c] = g;
    su[q][c] = u;
    __syncthreads();
    if (q == 0 && j < I) {
      g = sg[0][c] + sg[1][c] + sg[2][c] + sg[3][c];
      u = su[0][c] + su[1][c] + su[2][c] + su[3][c];
      hid[pair * I + j] = g / (1.0f + expf(-g)) * u;
    }
    __syncthreads();
  }
}

// y_t := sum_k p_k hid[t, k] W2[e_k] + beta y_t at 64 columns.
__global__ void __launch_bounds__(kThreads)
    moe_down_kernel(const float* __restrict__ hid, const uint16_t* __restrict__ W2,
                    const int* __restrict__ ids, const float* __restrict__ probs,
                    uint16_t* __restrict__ Y, long long ldy, int T, int H, int I, int topk,
                    float beta) {
  __shared__ float sy[4][64];
  const int tiles = (H + 63) / 64;
  const int c = threadIdx.x & 63, q = threadIdx.x >> 6;
  for (long long it = blockIdx.x; it < static_cast<long long>(T) * tiles; it += gridDim.x) {
    const long long t = it / tiles;
    const int j = static_cast<int>(it % tiles) * 64 + c;
    float y = 0.0f;
    if (j < H)
      for (int k = 0; k < topk; ++k) {
        const long long pair = t * topk + k;
        const uint16_t* w = W2 + static_cast<long long>(ids[pair]) * I * H + j;
        const float* h = hid + pair * I;
        float s = 0.0f;
        for (int i = q; i < I; i += 4) s = fmaf(h[i], h2f(w[static_cast<long long>(i) * H]), s);
        y = fmaf(probs[pair], s, y);
      }
    sy[q][c] = y;
    __syncthreads();
    if (q == 0 && j < H) {
      y = sy[0][c] + sy[1][c] + sy[2][c] + sy[3][c];
      uint16_t* o = Y + t * ldy + j;
      *o = f2h(beta != 0.0f ? fmaf(beta, h2f(*o), y) : y);
    }
    __syncthreads();
  }
}

int grid_for(long long items, int sms, int per_sm) {
  return static_cast<int>(std::max(1ll, std::min<long long>(items, 1ll * sms * per_sm)));
}

int status_of(cudaError_t e) {
  return counted_launch(e) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

int moe_any(const MoeArgs& m, int sms, cudaStream_t stream) {
  const size_t pairs = static_cast<size_t>(m.T) * m.topk;
  const size_t id_bytes = round256(4 * pairs), h_bytes = round256(4 * pairs * m.I);
  void* buf = nullptr;
  if (int rc = routed_scratch(stream, 2 * id_bytes + h_bytes, &buf)) return rc;
  uint8_t* const b = static_cast<uint8_t*>(buf);
  int* const ids = reinterpret_cast<int*>(b);
  float* const probs = reinterpret_cast<float*>(b + id_bytes);
  float* const hid = reinterpret_cast<float*>(b + 2 * id_bytes);
  moe_route_kernel<<<grid_for(m.T, sms, 8), kThreads, 0, stream>>>(
      m.X, m.ldx, m.Wr, m.T, m.H, m.E, m.topk, m.renormalize, ids, probs, m.ids, m.probs);
  if (int rc = status_of(cudaGetLastError())) return rc;
  if (m.I > 0) {
    const long long up = static_cast<long long>(pairs) * ((m.I + 63) / 64);
    moe_up_kernel<<<grid_for(up, sms, 8), kThreads, 0, stream>>>(m.X, m.ldx, m.W1, ids, hid, m.T,
                                                                 m.H, m.I, m.topk);
    if (int rc = status_of(cudaGetLastError())) return rc;
  }
  const long long down = 1ll * m.T * ((m.H + 63) / 64);
  moe_down_kernel<<<grid_for(down, sms, 8), kThreads, 0, stream>>>(
      hid, m.W2, ids, probs, m.Y, m.ldy, m.T, m.H, m.I, m.topk, m.beta);
  if (int rc = status_of(cudaGetLastError())) return rc;
  set_last_path("moe.any");
  return GEMM_OK;
}

}  // namespace
}  // namespace gb300

using namespace gb300;

extern "C" int gemm_f16_moe(const uint16_t* X, const uint16_t* Wr, const uint16_t* W1,
                            const uint16_t* W2, uint16_t* Y, int* ids, float* probs, int T, int H,
                            int I, int E, int topk, int renormalize, int ldx, int ldy, float beta,
                            cudaStream_t stream) {
  if (T < 0 || H < 0 || I < 0 || E < 0) return GEMM_ERR_DIM;
  if (T == 0 || H == 0) return GEMM_OK;
  if (E > kMaxExperts || topk < 1 || topk > E || topk > kMaxTopk) return GEMM_ERR_ARG;
  if (ldx < H || ldy < H) return GEMM_ERR_LD;
  if (!X || !Wr || !Y || (I > 0 && (!W1 || !W2))) return GEMM_ERR_NULL;
  const uintptr_t halves = reinterpret_cast<uintptr_t>(X) | reinterpret_cast<uintptr_t>(Wr) |
                           reinterpret_cast<uintptr_t>(W1) | reinterpret_cast<uintptr_t>(W2) |
                           reinterpret_cast<uintptr_t>(Y);
  const uintptr_t words = reinterpret_cast<uintptr_t>(ids) | reinterpret_cast<uintptr_t>(probs);
  if ((halves & 1u) || (words & 3u)) return GEMM_ERR_ARG;
  int sms = 0;
  DeviceStatus* st = nullptr;
  unsigned long long limit = 0;
  if (int rc = query_device(&sms, &st, &limit)) return rc;
  std::unique_lock<std::recursive_mutex> call;
  if (int rc = lock_stream(stream, &call)) return rc;
  const MoeArgs m{X, Wr, W1, W2, Y, ids, probs, T, H, I, E, topk, renormalize, ldx, ldy, beta};
  return moe_stream_fits(m) ? moe_stream(m, sms, st, limit, stream) : moe_any(m, sms, stream);
}
