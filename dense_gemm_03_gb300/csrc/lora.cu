// lora.cu -- a shared projection with low-rank adapters picked by row, and its
// gradients: argument checks, alignment copies and path choice.
//
//   forward    V_i = s[a] X_i A[a],  C_i := alpha (X_i W + V_i B[a]) + beta C_i
//   gradients  U_i = s[a] dC_i B[a]^T,
//              dX_i := alpha (dC_i W^T + U_i A[a]^T),
//              dA[a] := alpha sum_{i in a} X_i^T U_i + beta dA[a],
//              dB[a] := alpha sum_{i in a} V_i^T dC_i + beta dB[a]
// with a = ids[i]; a row whose id names no adapter (negative or >= adapters)
// has only the shared projection, and no adapter's weights touch it.
//
//   V and U     lora_shrink.cu on the tensor cores; lora_rows.cu for a few rows
//               forward, or few rows over many adapters
//   C and dX    lora_stream.cu where the result has few tiles; else the pair
//               kernel of gemm_f16_tc_kernel.cuh with the adapters as more
//               k-blocks of its tiles
//   dA and dB   lora_outer.cu
// V and U are fp32; every sum is fp32; C and dX are rounded once.
#include <cmath>
#include <initializer_list>

#include "lora.h"
#include "operands.h"

namespace gb300 {
namespace {

constexpr int kThreads = 256;

// G := beta * G over n floats (G := 0 when beta == 0, without reading it).
__global__ void __launch_bounds__(kThreads) scale_flat_kernel(float* __restrict__ G, long long n,
                                                              float beta) {
  for (long long i = blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x; i < n;
       i += static_cast<long long>(gridDim.x) * kThreads)
    G[i] = beta == 0.0f ? 0.0f : beta * G[i];
}

// Empty lists (n zeros) and M rows without an adapter.
__global__ void __launch_bounds__(kThreads) no_adapters_kernel(int* __restrict__ lists, int n,
                                                               int* __restrict__ ids, int M) {
  for (int i = blockIdx.x * kThreads + threadIdx.x; i < max(n, M); i += gridDim.x * kThreads) {
    if (i < n) lists[i] = 0;
    if (i < M) ids[i] = -1;
  }
}

int status_of(cudaError_t e) {
  return counted_launch(e) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

// What lora_shrink needs to know, apart from its jobs and its check.
LoraShrinkPlan shrink_plan(const LoraArgs& p) {
  LoraShrinkPlan s{};
  s.ids = p.ids;
  s.scales = p.scales;
  s.M = p.M;
  s.R = p.R;
  s.adapters = p.adapters;
  s.ldv = (p.R + 3) / 4 * 4;
  return s;
}

// See lora_shrink.cu on rows with small entries.
float large_weight(int R, float alpha) {
  return 1.0f / (std::fabs(alpha) * std::sqrt(static_cast<float>(R)));
}

int forward(LoraArgs p, uint16_t* C, int ldc, float alpha, float beta, const LoraDevice& d,
            cudaStream_t stream) {
  const bool chunks = lora_stream_suits(p.M, p.N, d.sms);
  const bool few = chunks && lora_stream_shrinks(p.M, p.K, p.R);   // the stream makes V itself
  // the pair kernel aligns W by itself
  Aligned x(p.X, p.ldx, p.M, p.K, true), w(p.W, p.ldw, p.K, p.N, chunks);
  Aligned a(p.A, p.lda, 1ll * p.adapters * p.K, p.R, true, few);
  Aligned b(p.B, p.ldb, 1ll * p.adapters * p.R, p.N, true);
  const size_t copies = x.bytes() + w.bytes() + a.bytes() + b.bytes();
  LoraShrinkPlan s = shrink_plan(p);
  LoraStream t{};
  auto describe = [&]() {   // of the operands as they are by now
    s.job[0] = LoraShrinkJob{p.X, p.ldx, p.K, p.A, p.lda, p.a_stride(), 0, chunks ? 0 : kLoraPacked};
    s.njobs = 1;
    s.max_c = p.K;
    s.sum_c = p.K;
    if (!chunks) {
      s.check = p.B;
      s.ld_check = p.ldb;
      s.check_stride = p.b_stride();
      s.check_rows = p.R;
      s.check_cols = p.N;
      s.large = large_weight(p.R, alpha);
    }
    t = LoraStream{p.X, p.W, C, p.ldx, p.ldw, ldc, p.M, p.N, p.K, p.R, p.adapters, 0, p.B, p.ldb,
                   p.b_stride(), nullptr, s.ldv, p.A, p.lda, p.a_stride(), p.ids, p.scales, alpha,
                   beta};
  };
  describe();
  void* buf = nullptr;
  const size_t shrink = few ? 0 : lora_shrink_bytes(s);
  const size_t need = copies + shrink + (chunks ? lora_stream_bytes(t, d.sms) : 0);
  if (int rc = routed_scratch(stream, need, &buf)) return rc;
  uint8_t* const rest = static_cast<uint8_t*>(buf) + copies;
  if (int rc = align_operands({{x, &p.X, &p.ldx}, {w, &p.W, &p.ldw}, {a, &p.A, &p.lda},
                               {b, &p.B, &p.ldb}},
                              static_cast<uint8_t*>(buf), d.sms, stream))
    return rc;
  describe();
  if (!few)
    if (int rc = lora_shrink(s, rest, d, stream)) return rc;
  if (chunks) {
    t.V = few ? nullptr : s.job[0].V;
    if (int rc = lora_stream(t, rest + shrink, d, stream)) return rc;
    set_last_path(copies ? "lora.stream.realigned" : "lora.stream");
    return GEMM_OK;
  }
  LoraCall call{};
  call.trans = false;
  call.tail = LoraTailArgs{s.job[0].V, s.job[0].packed, s.job[0].apart, s.ldv, p.ids, s.lists, s.bad,
                           p.B, p.ldb, p.b_stride(), p.R, p.adapters, (p.R + 31) / 32};
  if (int rc = gemm_f16_lora_pair(p.X, p.W, C, p.M, p.N, p.K, p.ldx, p.ldw, ldc, alpha, beta, call,
                                  stream))
    return rc;
  set_last_path(copies ? "lora.tiles.realigned" : "lora.tiles");
  return GEMM_OK;
}

int gradients(LoraArgs p, const uint16_t* G, int ldg, uint16_t* dX, int lddx, float* dA, float* dB,
              float alpha, float beta, const LoraDevice& d, cudaStream_t stream) {
  const bool use_u = dX || dA, use_v = dB != nullptr;
  const bool chunks = dX && lora_stream_suits(p.M, p.K, d.sms);
  // by rows where the result's dX (if any) does not need the lists of tiles;
  // the rule goes by sizes alone, so that a gradient asked for alone has the bits
  // it has beside the others
  LoraShrinkPlan rule = shrink_plan(p);
  rule.max_c = std::max(p.N, p.K);
  rule.sum_c = 1ll * p.N + p.K;
  const bool by_rows = lora_stream_suits(p.M, p.K, d.sms) && lora_rows_suit(rule);
  Aligned g(G, ldg, p.M, p.N, true), x(p.X, p.ldx, p.M, p.K, dA || dB);
  Aligned a(p.A, p.lda, 1ll * p.adapters * p.K, p.R, dX || dB, by_rows);
  Aligned b(p.B, p.ldb, 1ll * p.adapters * p.R, p.N, use_u);
  Aligned w(p.W, p.ldw, p.K, p.N, chunks);
  const size_t copies = g.bytes() + x.bytes() + a.bytes() + b.bytes() + w.bytes();
  LoraShrinkPlan s = shrink_plan(p);
  LoraStream t{};
  auto describe = [&]() {
    s.njobs = 0;
    s.max_c = std::max(p.N, p.K);
    s.sum_c = 1ll * p.N + p.K;
    if (use_u)
      s.job[s.njobs++] = LoraShrinkJob{G, ldg, p.N, p.B, p.ldb, p.b_stride(), 1,
                                       (dX && !chunks ? kLoraPacked : 0) | (dA ? kLoraScaled : 0)};
    if (use_v)
      s.job[s.njobs++] =
          LoraShrinkJob{p.X, p.ldx, p.K, p.A, p.lda, p.a_stride(), 0, kLoraScaled};
    if (dX && !chunks) {
      s.check = p.A;
      s.ld_check = p.lda;
      s.check_stride = p.a_stride();
      s.check_rows = p.K;
      s.check_cols = p.R;
      s.large = large_weight(p.R, alpha);
    }
    // any address for V: the stream makes none of its own
    t = LoraStream{G, p.W, dX, ldg, p.ldw, lddx, p.M, p.K, p.N, p.R, p.adapters, 1, p.A, p.lda,
                   p.a_stride(), p.scales ? p.scales : reinterpret_cast<const float*>(p.ids), s.ldv,
                   nullptr, 0, 0, p.ids, nullptr, alpha, 0.0f};
  };
  describe();
  LoraOuter o{p.X, G, p.ldx, ldg, nullptr, nullptr, p.ids, dA, dB, p.M, p.N, p.K, p.R,
              p.adapters, alpha, beta};
  const bool outer = dA || dB;
  const size_t shrink_bytes = by_rows ? lora_rows_bytes(s, d.sms) : lora_shrink_bytes(s);
  const size_t stream_bytes = chunks ? lora_round256(lora_stream_bytes(t, d.sms)) : 0;
  void* buf = nullptr;
  if (int rc = routed_scratch(stream, copies + shrink_bytes + stream_bytes +
                                          (outer ? lora_outer_bytes(o) : 0),
                              &buf))
    return rc;
  uint8_t* const rest = static_cast<uint8_t*>(buf) + copies;
  if (int rc = align_operands({{g, &G, &ldg}, {x, &p.X, &p.ldx}, {a, &p.A, &p.lda},
                               {b, &p.B, &p.ldb}, {w, &p.W, &p.ldw}},
                              static_cast<uint8_t*>(buf), d.sms, stream))
    return rc;
  describe();
  if (int rc = by_rows ? lora_rows(s, rest, d, stream) : lora_shrink(s, rest, d, stream)) return rc;
  if (chunks) {
    t.V = s.job[0].V;
    if (int rc = lora_stream(t, rest + shrink_bytes, d, stream)) return rc;
  } else if (dX) {
    LoraCall call{};
    call.trans = true;
    call.tail = LoraTailArgs{s.job[0].V, s.job[0].packed, s.job[0].apart, s.ldv, p.ids, s.lists,
                             s.bad, p.A, p.lda, p.a_stride(), p.R, p.adapters, (p.R + 31) / 32};
    if (int rc = gemm_f16_lora_pair(G, p.W, dX, p.M, p.K, p.N, ldg, p.ldw, lddx, alpha, 0.0f, call,
                                    stream))
      return rc;
  }
  if (outer) {
    o.X = p.X;
    o.ldx = p.ldx;
    o.G = G;
    o.ldg = ldg;
    o.U = dA ? &s.job[0] : nullptr;
    o.V = dB ? &s.job[s.njobs - 1] : nullptr;
    if (int rc = lora_outer(o, rest + shrink_bytes + stream_bytes, d, stream)) return rc;
  }
  set_last_path(chunks ? (copies ? "lora_grad.stream.realigned" : "lora_grad.stream")
                       : (copies ? "lora_grad.tiles.realigned" : "lora_grad.tiles"));
  return GEMM_OK;
}

// dX = alpha dC W^T alone (no adapters): the same kernel with empty lists.
int plain_dx(const LoraArgs& p, const uint16_t* G, int ldg, uint16_t* dX, int lddx, float alpha,
             const LoraDevice& d, cudaStream_t stream) {
  const int blocks = (p.M + 255) / 256;
  void* buf = nullptr;
  const size_t list_bytes = 4 * static_cast<size_t>(blocks) * kLoraListStride;
  if (int rc = routed_scratch(stream, lora_round256(list_bytes) + 4 * static_cast<size_t>(p.M), &buf))
    return rc;
  int* const lists = static_cast<int*>(buf);
  int* const none = reinterpret_cast<int*>(static_cast<uint8_t*>(buf) + lora_round256(list_bytes));
  no_adapters_kernel<<<d.sms, kThreads, 0, stream>>>(lists, blocks * kLoraListStride, none, p.M);
  if (int rc = status_of(cudaGetLastError())) return rc;
  LoraCall call{};
  call.trans = true;
  // any mapped matrix for the adapters' tensor map: no tile reads it
  const uint16_t* const any = reinterpret_cast<const uint16_t*>(buf);
  call.tail = LoraTailArgs{nullptr, any, nullptr, 4, none, lists, nullptr, any, 8, 8, 1, 1, 1};
  if (int rc = gemm_f16_lora_pair(G, p.W, dX, p.M, p.K, p.N, ldg, p.ldw, lddx, alpha, 0.0f, call,
                                  stream))
    return rc;
  set_last_path("lora_grad.plain");
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
  if (R > kLoraMaxRank) return GEMM_ERR_ARG;
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
  std::unique_lock<std::recursive_mutex> call;
  if (int rc = lock_stream(stream, &call)) return rc;
  const LoraArgs p{X, W, A, B, ids, scales, M, N, K, R, adapters, ldx, ldw, lda, ldb};
  return forward(p, C, ldc, alpha, beta, LoraDevice{sms, st, limit}, stream);
}

int gemm_f16_lora_grad(const uint16_t* dC, const uint16_t* X, const uint16_t* W, const uint16_t* A,
                       const uint16_t* B, const int* ids, const float* scales, uint16_t* dX,
                       float* dA, float* dB, int M, int N, int K, int R, int adapters, int lddc,
                       int ldx, int ldw, int lda, int ldb, int lddx, float alpha, float beta,
                       cudaStream_t stream) {
  if (M < 0 || N < 0 || K < 0 || R < 0 || adapters < 0) return GEMM_ERR_DIM;
  if (R > kLoraMaxRank || adapters > kLoraMaxAdapters) return GEMM_ERR_ARG;
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
  std::unique_lock<std::recursive_mutex> call;
  if (int rc = lock_stream(stream, &call)) return rc;
  const LoraArgs p{X, W, A, B, ids, scales, M, N, K, R, adapters, ldx, ldw, lda, ldb};
  const LoraDevice d{sms, st, limit};
  if (!grads) return plain_dx(p, dC, lddc, dX, lddx, alpha, d, stream);
  return gradients(p, dC, lddc, want_dx ? dX : nullptr, lddx, dA, dB, alpha, beta, d, stream);
}

}  // extern "C"
