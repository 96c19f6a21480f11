// lora.cu -- a shared projection with low-rank adapters picked by row, and its
// gradients: argument checks, path choice, and the CUDA-core kernels.
//
//   forward    V_i = s[a] X_i A[a],  C_i := alpha (X_i W + V_i B[a]) + beta C_i
//   gradients  U_i = s[a] dC_i B[a]^T,
//              dX_i := alpha (dC_i W^T + U_i A[a]^T),
//              dA[a] := alpha sum_{i in a} X_i^T U_i + beta dA[a],
//              dB[a] := alpha sum_{i in a} V_i^T dC_i + beta dB[a]
// with a = ids[i]; a row whose id names no adapter (negative or >= adapters)
// has only the shared projection, and no adapter's weights touch it.  V and U
// stay in fp32; every sum is fp32; C and dX are rounded once.
//
// The path of this file serves every alignment: the shared product is the
// library's half GEMM with a float result in scratch, and the kernels below
// add the low-rank part to it in fp32.
#include <initializer_list>

#include "lora.h"

namespace gb300 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxRank = kLoraMaxRank;

__device__ __forceinline__ float h2f(uint16_t b) { return lora_h2f(b); }
__device__ __forceinline__ uint16_t f2h(float x) { return lora_f2h(x); }

__device__ __forceinline__ float row_scale(const float* scales, int a) {
  return scales ? scales[a] : 1.0f;
}

// out[i][r] = s[a] * sum_c x_i[c] * F[a][c][r] (KMAJOR false: F rows run along
// the contraction, R values each, leading dimension ldf) or F[a][r][c] (KMAJOR
// true).  One block per row of x; a row without an adapter gets zeros.
template <bool KMAJOR>
__global__ void __launch_bounds__(kThreads)
    lora_shrink_kernel(const uint16_t* __restrict__ x, long long ldx,
                       const uint16_t* __restrict__ F, long long ldf, long long f_stride,
                       const int* __restrict__ ids, const float* __restrict__ scales,
                       float* __restrict__ out, int M, int C, int R, int adapters) {
  __shared__ float part[kWarps][kMaxRank];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = blockIdx.x; i < M; i += gridDim.x) {
    const int a = ids[i];
    float* const o = out + static_cast<long long>(i) * R;
    if (a < 0 || a >= adapters) {
      for (int r = threadIdx.x; r < R; r += kThreads) o[r] = 0.0f;
      continue;
    }
    const uint16_t* xi = x + static_cast<long long>(i) * ldx;
    const uint16_t* f = F + static_cast<long long>(a) * f_stride;
    if (KMAJOR) {
      for (int r = warp; r < R; r += kWarps) {
        const uint16_t* fr = f + static_cast<long long>(r) * ldf;
        float s = 0.0f;
        for (int c = lane; c < C; c += 32) s = fmaf(h2f(xi[c]), h2f(fr[c]), s);
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        if (lane == 0) o[r] = row_scale(scales, a) * s;
      }
    } else {
      float acc[kMaxRank / 32] = {};
      for (int c = warp; c < C; c += kWarps) {
        const float xv = h2f(xi[c]);
        const uint16_t* fc = f + static_cast<long long>(c) * ldf;
#pragma unroll
        for (int q = 0; q < kMaxRank / 32; ++q)
          if (lane + 32 * q < R) acc[q] = fmaf(xv, h2f(fc[lane + 32 * q]), acc[q]);
      }
#pragma unroll
      for (int q = 0; q < kMaxRank / 32; ++q) part[warp][lane + 32 * q] = acc[q];
      __syncthreads();
      for (int r = threadIdx.x; r < R; r += kThreads) {
        float s = 0.0f;
        for (int w = 0; w < kWarps; ++w) s += part[w][r];
        o[r] = row_scale(scales, a) * s;
      }
      __syncthreads();
    }
  }
}

// C_i := alpha (D_i + v_i F[a]) + beta C_i, with F[a][r][c] (TRANS false) or
// F[a][c][r] (TRANS true).  One block per (row, 1024 columns).
template <bool TRANS>
__global__ void __launch_bounds__(kThreads)
    lora_expand_kernel(const float* __restrict__ D, long long ldd, const float* __restrict__ v,
                       const uint16_t* __restrict__ F, long long ldf, long long f_stride,
                       const int* __restrict__ ids, uint16_t* __restrict__ C, long long ldc, int M,
                       int N, int R, int adapters, float alpha, float beta) {
  __shared__ float vs[kMaxRank];
  const int chunks = (N + 4 * kThreads - 1) / (4 * kThreads);
  const long long items = static_cast<long long>(M) * chunks;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int i = static_cast<int>(it / chunks);
    const int c0 = static_cast<int>(it % chunks) * 4 * kThreads;
    const int a = R > 0 ? ids[i] : -1;
    const bool has = a >= 0 && a < adapters;
    __syncthreads();
    for (int r = threadIdx.x; r < R; r += kThreads) vs[r] = v[static_cast<long long>(i) * R + r];
    __syncthreads();
    const uint16_t* f = F + (has ? static_cast<long long>(a) * f_stride : 0);
    for (int j = 0; j < 4; ++j) {
      const int c = c0 + j * kThreads + threadIdx.x;
      if (c >= N) break;
      float s = 0.0f;
      if (has)
        for (int r = 0; r < R; ++r)
          s = fmaf(vs[r],
                   h2f(TRANS ? f[static_cast<long long>(c) * ldf + r]
                             : f[static_cast<long long>(r) * ldf + c]),
                   s);
      s += D[static_cast<long long>(i) * ldd + c];
      uint16_t* o = C + static_cast<long long>(i) * ldc + c;
      *o = f2h(beta != 0.0f ? fmaf(alpha, s, beta * h2f(*o)) : alpha * s);
    }
  }
}

// G[a] (rows x cols of a stack, row stride ldg) := alpha * sum over the rows i
// of adapter a of y_i (outer) x_i + beta * G[a].  XROWS true: G[a][c][r] =
// sum x_i[c] y_i[r] (dA: x = X, y = U); false: G[a][r][c] (dB: x = dC, y = V).
// One block per (adapter, 32 columns c): thread (c, q) holds ranks q, q + 8, ...
template <bool XROWS>
__global__ void __launch_bounds__(kThreads)
    lora_outer_kernel(const uint16_t* __restrict__ x, long long ldx, const float* __restrict__ y,
                      const int* __restrict__ ids, float* __restrict__ G, int M, int C, int R,
                      int adapters, float alpha, float beta) {
  __shared__ int rows[kThreads];
  __shared__ int count[kWarps];
  constexpr int kPer = kMaxRank / kWarps;
  const int tiles = (C + 31) / 32;
  const int lane = threadIdx.x & 31, q = threadIdx.x >> 5;
  for (long long it = blockIdx.x; it < static_cast<long long>(adapters) * tiles; it += gridDim.x) {
    const int a = static_cast<int>(it / tiles);
    const int c = static_cast<int>(it % tiles) * 32 + lane;
    float acc[kPer] = {};
    for (int i0 = 0; i0 < M; i0 += kThreads) {
      // the rows of adapter a among these 256, in order
      const int i = i0 + static_cast<int>(threadIdx.x);
      const bool mine = i < M && ids[i] == a;
      const unsigned int ball = __ballot_sync(0xffffffffu, mine);
      __syncthreads();
      if (lane == 0) count[q] = __popc(ball);
      __syncthreads();
      int before = 0, total = 0;
      for (int w = 0; w < kWarps; ++w) {
        if (w < q) before += count[w];
        total += count[w];
      }
      if (mine) rows[before + __popc(ball & ((1u << lane) - 1u))] = i;
      __syncthreads();
      for (int k = 0; k < total; ++k) {
        const long long row = rows[k];
        const float xv = c < C ? h2f(x[row * ldx + c]) : 0.0f;
#pragma unroll
        for (int p = 0; p < kPer; ++p)
          if (q + kWarps * p < R) acc[p] = fmaf(xv, y[row * R + q + kWarps * p], acc[p]);
      }
    }
    if (c < C) {
      float* g = G + static_cast<long long>(a) * C * R;
#pragma unroll
      for (int p = 0; p < kPer; ++p) {
        const int r = q + kWarps * p;
        if (r < R) {
          float* o = g + (XROWS ? static_cast<long long>(c) * R + r
                                : static_cast<long long>(r) * C + c);
          *o = beta != 0.0f ? fmaf(alpha, acc[p], beta * *o) : alpha * acc[p];
        }
      }
    }
  }
}

// dst (cols x rows, leading dimension ldd) := transpose of src (rows x cols).
__global__ void __launch_bounds__(kThreads)
    transpose_f16_kernel(const uint16_t* __restrict__ src, long long lds, uint16_t* __restrict__ dst,
                         long long ldd, int rows, int cols) {
  __shared__ uint16_t tile[32][33];
  const int tc = (cols + 31) / 32;
  const long long tiles = static_cast<long long>((rows + 31) / 32) * tc;
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  for (long long t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int r0 = static_cast<int>(t / tc) * 32, c0 = static_cast<int>(t % tc) * 32;
    __syncthreads();
    for (int j = y; j < 32; j += kWarps)
      if (r0 + j < rows && c0 + x < cols)
        tile[j][x] = src[static_cast<long long>(r0 + j) * lds + c0 + x];
    __syncthreads();
    for (int j = y; j < 32; j += kWarps)
      if (c0 + j < cols && r0 + x < rows)
        dst[static_cast<long long>(c0 + j) * ldd + r0 + x] = tile[x][j];
  }
}

// G := beta * G over n floats (G := 0 when beta == 0, without reading it).
__global__ void __launch_bounds__(kThreads) scale_flat_kernel(float* __restrict__ G, long long n,
                                                              float beta) {
  for (long long i = blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x; i < n;
       i += static_cast<long long>(gridDim.x) * kThreads)
    G[i] = beta == 0.0f ? 0.0f : beta * G[i];
}

int grid_for(long long items, int sms, int per_sm) {
  return static_cast<int>(std::max(1ll, std::min<long long>(items, 1ll * sms * per_sm)));
}

int status_of(cudaError_t e) {
  return counted_launch(e) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

size_t round256(size_t x) { return lora_round256(x); }

bool on16(const void* p, long long ld) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 8 == 0;
}

bool misaligned(std::initializer_list<const void*> ptrs, size_t elem) {
  uintptr_t bits = 0;
  for (const void* p : ptrs) bits |= reinterpret_cast<uintptr_t>(p);
  return (bits & (elem - 1)) != 0;
}

int forward_any(const LoraArgs& p, uint16_t* C, int ldc, float alpha, float beta, int sms,
                cudaStream_t stream) {
  const long long ldd = (p.N + 3) / 4 * 4;
  const size_t d_bytes = round256(sizeof(float) * static_cast<size_t>(p.M) * ldd);
  const size_t v_bytes = round256(sizeof(float) * static_cast<size_t>(p.M) * p.R);
  void* buf = nullptr;
  if (int rc = routed_scratch(stream, d_bytes + v_bytes, &buf)) return rc;
  float* const D = static_cast<float*>(buf);
  float* const V = reinterpret_cast<float*>(static_cast<uint8_t*>(buf) + d_bytes);
  lora_shrink_kernel<false><<<grid_for(p.M, sms, 8), kThreads, 0, stream>>>(
      p.X, p.ldx, p.A, p.lda, p.a_stride(), p.ids, p.scales, V, p.M, p.K, p.R, p.adapters);
  if (int rc = status_of(cudaGetLastError())) return rc;
  if (int rc = gemm_f16_f32out(p.X, p.W, D, p.M, p.N, p.K, p.ldx, p.ldw, static_cast<int>(ldd),
                               1.0f, 0.0f, stream))
    return rc;
  const long long items = 1ll * p.M * ((p.N + 4 * kThreads - 1) / (4 * kThreads));
  lora_expand_kernel<false><<<grid_for(items, sms, 8), kThreads, 0, stream>>>(
      D, ldd, V, p.B, p.ldb, p.b_stride(), p.ids, C, ldc, p.M, p.N, p.R, p.adapters, alpha, beta);
  if (int rc = status_of(cudaGetLastError())) return rc;
  set_last_path("lora.any");
  return GEMM_OK;
}

// Many rows: the low-rank products on the tensor cores, then the pair kernel
// with the adapters as more k-blocks of its tiles.
int forward_tiles(const LoraArgs& p, uint16_t* C, int ldc, float alpha, float beta,
                  const LoraDevice& d, cudaStream_t stream) {
  LoraShrinkPlan s{};
  s.job[0] = LoraShrinkJob{p.X, p.ldx, p.K, p.A, p.lda, p.a_stride(), 0, nullptr, 0};
  s.njobs = 1;
  s.ids = p.ids;
  s.scales = p.scales;
  s.M = p.M;
  s.R = p.R;
  s.adapters = p.adapters;
  s.ldv = (p.R + 3) / 4 * 4;
  s.check = p.B;
  s.ld_check = p.ldb;
  s.check_stride = p.b_stride();
  s.check_rows = p.R;
  s.check_cols = p.N;
  void *buf = nullptr, *zero = nullptr;
  if (int rc = routed_scratch(stream, lora_shrink_bytes(s, d.sms), &buf,
                              4 * 8 * static_cast<size_t>((p.M + 127) / 128), &zero))
    return rc;
  if (int rc = lora_shrink(s, buf, static_cast<unsigned int*>(zero), d, stream)) return rc;
  LoraCall call{};
  call.trans = false;
  call.tail = LoraTailArgs{s.job[0].V, s.ldv, p.ids, s.lists, s.bad, p.B, p.ldb, p.b_stride(),
                           p.R, p.adapters, (p.R + 31) / 32};
  if (int rc = gemm_f16_lora_pair(p.X, p.W, C, p.M, p.N, p.K, p.ldx, p.ldw, ldc, alpha, beta, call,
                                  stream))
    return rc;
  set_last_path("lora.tiles");
  return GEMM_OK;
}

int grad_any(const LoraArgs& p, const uint16_t* dC, int lddc, uint16_t* dX, int lddx, float* dA,
             float* dB, float alpha, float beta, int sms, cudaStream_t stream) {
  const long long ldd = (p.K + 3) / 4 * 4, ldt = (p.K + 7) / 8 * 8;
  const size_t v_bytes = round256(sizeof(float) * static_cast<size_t>(p.M) * p.R);
  const size_t d_bytes = dX ? round256(sizeof(float) * static_cast<size_t>(p.M) * ldd) : 0;
  const size_t t_bytes = dX ? round256(2 * static_cast<size_t>(p.N) * ldt) : 0;
  void* buf = nullptr;
  if (int rc = routed_scratch(stream, 2 * v_bytes + d_bytes + t_bytes, &buf)) return rc;
  uint8_t* const b = static_cast<uint8_t*>(buf);
  float* const V = reinterpret_cast<float*>(b);
  float* const U = reinterpret_cast<float*>(b + v_bytes);
  float* const D = reinterpret_cast<float*>(b + 2 * v_bytes);
  uint16_t* const Wt = reinterpret_cast<uint16_t*>(b + 2 * v_bytes + d_bytes);
  const int g_rows = grid_for(p.M, sms, 8);
  if ((dX || dA) && p.R > 0) {
    lora_shrink_kernel<true><<<g_rows, kThreads, 0, stream>>>(
        dC, lddc, p.B, p.ldb, p.b_stride(), p.ids, p.scales, U, p.M, p.N, p.R, p.adapters);
    if (int rc = status_of(cudaGetLastError())) return rc;
  }
  if (dB) {
    lora_shrink_kernel<false><<<g_rows, kThreads, 0, stream>>>(
        p.X, p.ldx, p.A, p.lda, p.a_stride(), p.ids, p.scales, V, p.M, p.K, p.R, p.adapters);
    if (int rc = status_of(cudaGetLastError())) return rc;
    lora_outer_kernel<false>
        <<<grid_for(1ll * p.adapters * ((p.N + 31) / 32), sms, 8), kThreads, 0, stream>>>(
            dC, lddc, V, p.ids, dB, p.M, p.N, p.R, p.adapters, alpha, beta);
    if (int rc = status_of(cudaGetLastError())) return rc;
  }
  if (dA) {
    lora_outer_kernel<true>
        <<<grid_for(1ll * p.adapters * ((p.K + 31) / 32), sms, 8), kThreads, 0, stream>>>(
            p.X, p.ldx, U, p.ids, dA, p.M, p.K, p.R, p.adapters, alpha, beta);
    if (int rc = status_of(cudaGetLastError())) return rc;
  }
  if (dX) {
    const long long tiles = 1ll * ((p.K + 31) / 32) * ((p.N + 31) / 32);
    transpose_f16_kernel<<<grid_for(tiles, sms, 8), kThreads, 0, stream>>>(p.W, p.ldw, Wt, ldt,
                                                                          p.K, p.N);
    if (int rc = status_of(cudaGetLastError())) return rc;
    if (int rc = gemm_f16_f32out(dC, Wt, D, p.M, p.K, p.N, lddc, static_cast<int>(ldt),
                                 static_cast<int>(ldd), 1.0f, 0.0f, stream))
      return rc;
    const long long items = 1ll * p.M * ((p.K + 4 * kThreads - 1) / (4 * kThreads));
    lora_expand_kernel<true><<<grid_for(items, sms, 8), kThreads, 0, stream>>>(
        D, ldd, U, p.A, p.lda, p.a_stride(), p.ids, dX, lddx, p.M, p.K, p.R, p.adapters, alpha,
        0.0f);
    if (int rc = status_of(cudaGetLastError())) return rc;
  }
  set_last_path("lora_grad.any");
  return GEMM_OK;
}

}  // namespace
}  // namespace gb300

using namespace gb300;

extern "C" {

int gemm_f16_lora(const uint16_t* X, const uint16_t* W, uint16_t* C, const uint16_t* A,
                  const uint16_t* B, const int* ids, const float* scales, int M, int N, int K,
                  int R, int adapters, int ldx, int ldw, int ldc, int lda, int ldb, float alpha,
                  float beta, cudaStream_t stream) {
  if (M < 0 || N < 0 || K < 0 || R < 0 || adapters < 0) return GEMM_ERR_DIM;
  if (R > kMaxRank) return GEMM_ERR_ARG;
  // nothing to add: the shared projection alone
  if (R == 0 || adapters == 0 || M == 0 || N == 0 || K == 0 || alpha == 0.0f)
    return gemm_f16_ld(X, W, C, M, N, K, ldx, ldw, ldc, alpha, beta, stream);
  if (ldx < K || ldw < N || ldc < N || lda < R || ldb < N) return GEMM_ERR_LD;
  if (!X || !W || !C || !A || !B || !ids) return GEMM_ERR_NULL;
  if (misaligned({X, W, C, A, B}, 2) || misaligned({ids, scales}, 4)) return GEMM_ERR_ARG;
  int sms = 0;
  DeviceStatus* st = nullptr;
  unsigned long long limit = 0;
  if (int rc = query_device(&sms, &st, &limit)) return rc;
  const LoraArgs p{X, W, A, B, ids, scales, M, N, K, R, adapters, ldx, ldw, lda, ldb};
  const LoraDevice d{sms, st, limit};
  // TMA and 16-byte loads want every operand's rows on the 16-byte grid, and
  // the ranks in groups of eight
  if (M <= kLoraStreamRows && R % 8 == 0 && on16(X, ldx) && on16(W, ldw) && on16(A, lda) &&
      on16(B, ldb))
    return lora_stream(p, C, ldc, alpha, beta, d, stream);
  if (M > kLoraStreamRows && N > 128 && on16(X, ldx) && on16(W, ldw) && on16(A, lda) && on16(B, ldb))
    return forward_tiles(p, C, ldc, alpha, beta, d, stream);
  return forward_any(p, C, ldc, alpha, beta, sms, stream);
}

int gemm_f16_lora_grad(const uint16_t* dC, const uint16_t* X, const uint16_t* W, const uint16_t* A,
                       const uint16_t* B, const int* ids, const float* scales, uint16_t* dX,
                       float* dA, float* dB, int M, int N, int K, int R, int adapters, int lddc,
                       int ldx, int ldw, int lda, int ldb, int lddx, float alpha, float beta,
                       cudaStream_t stream) {
  if (M < 0 || N < 0 || K < 0 || R < 0 || adapters < 0) return GEMM_ERR_DIM;
  if (R > kMaxRank) return GEMM_ERR_ARG;
  const bool grads = R > 0 && adapters > 0;   // dA and dB have elements
  const bool want_dx = dX != nullptr && M > 0 && K > 0;
  if (!grads) dA = dB = nullptr;
  if (K == 0) dA = nullptr;
  if (N == 0) dB = nullptr;
  if (!want_dx && !dA && !dB) return GEMM_OK;
  // does any product of M, N and K remain (else every result is beta times
  // its old value, and zero for dX)
  const bool some = M > 0 && N > 0 && K > 0 && alpha != 0.0f;
  if (want_dx && lddx < K) return GEMM_ERR_LD;
  if (some) {
    // dX reads dC, W, A, B; dA reads dC, X, B; dB reads dC, X, A
    const bool use_a = grads && (want_dx || dB), use_b = grads && (want_dx || dA);
    if (lddc < N || ((dA || dB) && ldx < K) || (want_dx && ldw < N) || (use_a && lda < R) ||
        (use_b && ldb < N))
      return GEMM_ERR_LD;
    if (!dC || ((dA || dB) && !X) || (want_dx && !W) || (use_a && !A) || (use_b && !B) ||
        (grads && !ids))
      return GEMM_ERR_NULL;
  }
  if (misaligned({dC, X, W, A, B, dX}, 2) || misaligned({ids, scales, dA, dB}, 4))
    return GEMM_ERR_ARG;
  int sms = 0;
  DeviceStatus* st = nullptr;
  unsigned long long limit = 0;
  if (int rc = query_device(&sms, &st, &limit)) return rc;
  if (!some) {
    set_last_path("lora_grad.scale");
    const int g = 8 * sms;
    if (want_dx && launch_scale_f16(dX, lddx, M, K, 0.0f, g, stream) != cudaSuccess)
      return GEMM_ERR_CUDA;
    const long long n_a = 1ll * adapters * K * R, n_b = 1ll * adapters * R * N;
    if (dA) {
      scale_flat_kernel<<<g, kThreads, 0, stream>>>(dA, n_a, beta);
      if (int rc = status_of(cudaGetLastError())) return rc;
    }
    if (dB) {
      scale_flat_kernel<<<g, kThreads, 0, stream>>>(dB, n_b, beta);
      if (int rc = status_of(cudaGetLastError())) return rc;
    }
    return GEMM_OK;
  }
  LoraArgs p{X, W, A, B, ids, scales, M, N, K, R, adapters, ldx, ldw, lda, ldb};
  if (!grads) {   // dX = alpha dC W^T: no row has an adapter
    p.R = p.adapters = 0;
  }
  return grad_any(p, dC, lddc, want_dx ? dX : nullptr, lddx, dA, dB, alpha, beta, sms, stream);
}

}  // extern "C"
