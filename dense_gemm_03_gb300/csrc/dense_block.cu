// dense_block.cu -- the gated block of a dense model, its gradients, and products
// with transposed operands: argument checks, alignment copies and path choice.
//
//   glu       C := f(X Wg) .* (X Wu),  W = [Wg Wu]
//   gradient  G = X Wg and U = X Wu again (one gated product whose epilogue reads dC),
//             dG = dC .* U .* f'(G), dU = dC .* f(G), dGU = [dG dU];
//             dX := dGU W^T, dW := X^T dGU + beta dW
//   trans     C := alpha op(A) op(B) + beta C
//
// Two ways for each product: whole 256 x 256 tiles on CTA pairs
// (gemm_f16_tc_kernel.cuh), or, where a few rows or few tiles would leave SMs idle,
// K cut into chunks (narrow_stream.cu).  Sums are fp32; every result is rounded once.
// dX and dW are products of dGU as it was rounded, where a chain that kept dGU in 32 bits would
// be 1.4 times nearer to 64 bits (errors of 2.9e-4 and 2.1e-4 of their norm): dGU in half is an
// output that the backward chain reads anyway, and the tensor cores take no wider operands at this
// rate (two halves each would double both products).
#include "gemm.h"
#include "lora.h"
#include "operands.h"
#include "stream.h"

namespace gb300 {
namespace {

bool known_act(int act) {
  return act == GEMM_ACT_SILU || act == GEMM_ACT_GELU || act == GEMM_ACT_GELU_TANH ||
         act == GEMM_ACT_RELU;
}

int blank(uint16_t* C, long long ldc, int M, int N, float beta, const LoraDevice& d,
          cudaStream_t stream) {
  return launch_scale_f16(C, ldc, M, N, beta, 8 * d.sms, stream) == cudaSuccess ? GEMM_OK
                                                                               : GEMM_ERR_CUDA;
}

// The streamed form: op(X) op(W) with `cols` columns, then the sum `s` (its parts are
// filled in here).
int streamed(const uint16_t* X, int ldx, bool trans_x, const uint16_t* W, int ldw, bool trans_w,
             int M, int cols, int K, StreamSum s, const PairDone* before, const LoraDevice& d,
             cudaStream_t stream, bool* copied) {
  Aligned x(X, ldx, trans_x ? K : M, trans_x ? M : K, true);
  Aligned w(W, ldw, trans_w ? cols : K, trans_w ? K : cols, true);
  const size_t copies = x.bytes() + w.bytes();
  NarrowStream p{X, W, ldx, ldw, K, trans_x, trans_w};
  const bool cluster = narrow_cluster_suits(p, s, d);
  if (!cluster) s.parts = narrow_parts(p, M, cols, s.f32 || s.fold, d);
  void* buf = nullptr;
  if (copies + s.parts.bytes)
    if (int rc = routed_scratch(stream, copies + s.parts.bytes, &buf)) return rc;
  if (int rc = align_operands({{x, &X, &ldx}, {w, &W, &ldw}}, static_cast<uint8_t*>(buf), d.sms,
                              stream, true))
    return rc;
  *copied = copies != 0;
  p = NarrowStream{X, W, ldx, ldw, K, trans_x, trans_w, before && before->pair && !*copied};
  if (cluster) return narrow_cluster(p, s, d, stream);
  s.parts.part = reinterpret_cast<float*>(static_cast<uint8_t*>(buf) + copies);
  if (int rc = narrow_partial(p, M, cols, s.f32 || s.fold, s.parts, d, stream)) return rc;
  return stream_sum(s, d, stream);
}

// Folded sums (`fold`) come as a chunk for each kFoldDepth of K: once these pass the L2, as many bytes again twice
// over HBM, and scratch.  Tiles that fold in registers take about 0.35 us a k-block and wave, chunks 5.9 TB/s:
// float results of 192 x 16384 over 16384, 403 MB of partial sums, 225 us, tiles 100; relu's gradient of 128 x 8192 x
// 2*8192, 134 MB, 90, 61; draws at 134 MB of 128 x 16384 x 2*4096 and 537 of 128 x 8192 over 65536; but 67 MB of
// 128 x 8192 over 8192 40, 49, and 34 of 128 x 1024 over 32768 28, 166.
bool folds_in_tiles(int M, int cols, int K, int sms) {
  const double part = 4.0 * M * cols * ((K + kFoldDepth - 1) / kFoldDepth);
  if (K <= kFoldDepth || part <= 96e6) return false;
  const long long tiles = ((M + 255ll) / 256) * ((cols + 255ll) / 256), pairs = sms / 2;
  return 0.35 * ((tiles + pairs - 1) / pairs) * ((K + 63) / 64) <
         (2.0 * K * (1.0 * M + cols) + 2 * part) / 5.9e6;
}

// Whether K chunks suit the product better than whole 256 x 256 tiles (`cols` columns of
// W).  Measured, chunks against tiles: a block of up to 128 rows wins or draws (128 x 8192
// x 2048 11.1 us, 14.4; 128 x 4096 x 512 6.2, 6.2), up to 192 with a sum long enough (160 x 4096 x
// 768 7.0, 7.3, but 192 x 4096 x 512 7.2, 6.2; 192 x 8192 x 2048 14.2, 14.5, but 224 rows 15.4,
// 14.6); so do few tiles with a long K (512 x 512 x 1536 9.5, 10.5; 331 x 2048 x 4096 11.7, 21.9; but
// 1024^3 9.3, 8.4, and 32 tiles, 1024 x 2048 x 2048, 14.4, 13.8) and narrow results (6000 x 128 x
// 1536 10.3, 11.0, 9000 x 64 x 1024 8.6, 8.8, but 2048 x 128 x 512 8.0, 6.1).
bool narrow_suits(int M, int cols, int K, bool fold, int sms) {
  if (fold && folds_in_tiles(M, cols, K, sms)) return false;
  if (M <= 128) return true;
  if (M <= 192) return K >= 768;
  const long long tiles = static_cast<long long>((M + 255) / 256) * ((cols + 255) / 256);
  return cols <= 128 ? 4 * tiles <= sms && K >= 1024 : 8 * tiles <= sms && K >= 1536;
}

// relu's derivative jumps at 0, where a sum's error turns dC U into nothing or back.
// The tensor core's additions truncate, and long sums of G drift further than sums
// rounded to nearest; so a relu's gradient over more than 1024 products adds up runs of
// kFoldDepth in fp32, in the tiles' registers or as the stream's chunks.
bool folds(int gate, int act, int K) { return gate == 2 && act == GEMM_ACT_RELU && K > 1024; }

struct GluArgs {
  const uint16_t *X, *W;
  int M, N, K, ldx, ldw, act;
  int up;   // U's columns come so many after G's, in W and in dGU (tiles: N or more)
};

// gate 1: C := f(G) .* U; gate 2: C = dGU.
int gated(const GluArgs& p, int gate, uint16_t* C, int ldc, const uint16_t* dC, int lddc,
          const LoraDevice& d, cudaStream_t stream) {
  GateArgs g{};
  g.act = p.act;
  g.up = p.up;
  g.dC = dC;
  g.lddc = lddc;
  g.dU = gate == 2 ? C + p.up : nullptr;
  const bool fold = folds(gate, p.act, p.K);
  if (narrow_suits(p.M, 2 * p.N, p.K, fold, d.sms)) {
    StreamSum s{};
    s.fold = fold;
    s.C = C;
    s.ldc = ldc;
    s.M = p.M;
    s.N = p.N;
    s.gate = gate;
    s.g = g;
    bool copied = false;
    if (int rc = streamed(p.X, p.ldx, false, p.W, p.ldw, false, p.M, 2 * p.N, p.K, s, nullptr, d,
                          stream, &copied))
      return rc;
    set_last_path(copied ? "glu.stream.realigned" : "glu.stream");
    return GEMM_OK;
  }
  PairCall q{};
  q.A = p.X;
  q.B = p.W;
  q.C = C;
  q.M = p.M;
  q.N = p.N;
  q.K = p.K;
  q.lda = p.ldx;
  q.ldb = p.ldw;
  q.ldc = ldc;
  q.alpha = 1.0f;
  q.gate = gate;
  q.fold = fold;
  q.g = g;
  return gemm_f16_pair(q, stream);
}

// C := alpha op(A) op(B) + beta C, checked, with M, N, K > 0 and alpha != 0.
struct Trans {
  const uint16_t *A, *B;
  void* C;
  bool f32, ta, tb;
  int M, N, K, lda, ldb, ldc;
  float alpha, beta;
  bool c_padded = false;   // see PairCall
  bool tiled(int sms) const { return !narrow_suits(M, N, K, f32, sms); }
  bool on_grid() const {   // no copies of the operands
    return !misaligned({A, B}, 16) && lda % 8 == 0 && ldb % 8 == 0;
  }
  bool c_on_grid() const {
    return f32 || (!misaligned({C}, 16) && ldc % 8 == 0 && (N % 8 == 0 || c_padded));
  }
  long long tiles() const { return 1ll * ((M + 255) / 256) * ((N + 255) / 256); }
};

// whole, most_pairs, before, done: see PairCall.
int transposed(const Trans& p, bool whole, int most_pairs, const PairDone* before, PairDone* done,
               const LoraDevice& d, cudaStream_t stream) {
  if (!p.tiled(d.sms)) {
    StreamSum s{};
    s.C = p.C;
    s.ldc = p.ldc;
    s.M = p.M;
    s.N = p.N;
    s.alpha = p.alpha;
    s.beta = p.beta;
    s.f32 = p.f32;
    bool copied = false;
    if (int rc = streamed(p.A, p.lda, p.ta, p.B, p.ldb, p.tb, p.M, p.N, p.K, s, before, d, stream,
                          &copied))
      return rc;
    set_last_path(copied ? "trans.stream.realigned" : "trans.stream");
    return GEMM_OK;
  }
  PairCall q{};
  q.A = p.A;
  q.B = p.B;
  q.C = p.C;
  q.c_f32 = p.f32;
  q.M = p.M;
  q.N = p.N;
  q.K = p.K;
  q.lda = p.lda;
  q.ldb = p.ldb;
  q.ldc = p.ldc;
  q.alpha = p.alpha;
  q.beta = p.beta;
  q.trans_a = p.ta;
  q.trans_b = p.tb;
  q.c_padded = p.c_padded;
  q.whole = whole;
  q.pairs = most_pairs;
  q.before = before;
  q.done = done;
  return gemm_f16_pair(q, stream);
}

// Two products of one call's operands.  Side by side (see PairDone) where one leaves
// enough SMs idle: whole tiles of that, the other on the SMs left, in as many rounds as it
// takes; k-blocks of the longer way are weighed against one after the other over all SMs, a
// kernel's start and end counting as 12.  Gradients of 1500 x 1000 x 2*1368, 24 tiles of 43
// k-blocks and 44 of 24: 48.2 us one after the other, 40.8 side by side; 4096 x 1024 x 2*1024, 32
// of 64 and 64 of 32: 66.3 and 52.6; 300 x 1000 x 2*1368, 44 of 5 and a streamed product: 32.2
// and 28.3.  Else the second starts as the first's last blocks end.
int both(const Trans& a, const Trans& b, const LoraDevice& d, cudaStream_t stream) {
  const bool ta = a.tiled(d.sms), tb = b.tiled(d.sms);
  // tiles before a streamed product, longer tiles before shorter ones
  const bool swap = ta != tb ? tb : b.K > a.K;
  const Trans &x = swap ? b : a, &y = swap ? a : b;
  const long long pairs = d.sms / 2, left = pairs - x.tiles();
  bool beside = (ta || tb) && left > 0 && x.c_on_grid() && y.on_grid() && y.c_on_grid();
  if (beside && ta && tb) {
    auto way = [](const Trans& t, long long on) {
      return static_cast<double>((t.tiles() + on - 1) / on) * ((t.K + 63) / 64);
    };
    auto alone = [&](const Trans& t) { return way(t, pairs) * (2 * t.tiles() <= pairs ? 0.75 : 1.0); };
    beside = std::max(way(x, pairs), way(y, left)) < alone(x) + alone(y) + 12;
  }
  PairDone done{};
  if (!beside) {
    if (int rc = transposed(a, false, 0, nullptr, &done, d, stream)) return rc;
    return transposed(b, false, 0, &done, nullptr, d, stream);
  }
  if (int rc = transposed(x, true, 0, nullptr, &done, d, stream)) return rc;
  return transposed(y, false, static_cast<int>(left), &done, nullptr, d, stream);
}

struct GradArgs {
  const uint16_t *dC, *X, *W;
  uint16_t *dGU, *dX, *dW;   // dX, dW: NULL when not wanted
  int M, N, K, act, lddc, ldx, ldw, lddgu, lddx, lddw;
  int up;                    // as in GluArgs; dX and dW are products with all 2 up columns
  float beta;
  bool dx_padded = false;    // columns of dX up to a multiple of eight may be written
};

int grad_products(const GradArgs& p, const LoraDevice& d, cudaStream_t stream) {
  if (int rc = gated(GluArgs{p.X, p.W, p.M, p.N, p.K, p.ldx, p.ldw, p.act, p.up}, 2, p.dGU, p.lddgu,
                     p.dC, p.lddc, d, stream))
    return rc;
  const int cols = 2 * p.up;
  const Trans dx{p.dGU, p.W, p.dX, false, false, true, p.M, p.K, cols, p.lddgu, p.ldw, p.lddx, 1.0f, 0.0f,
                 p.dx_padded};
  const Trans dw{p.X, p.dGU, p.dW, false, true, false, p.K, cols, p.M, p.ldx, p.lddgu, p.lddw, 1.0f, p.beta};
  if (p.dX && p.dW) return both(dx, dw, d, stream);
  if (!p.dX && !p.dW) return GEMM_OK;
  return transposed(p.dX ? dx : dw, false, 0, nullptr, nullptr, d, stream);
}

// Matrices that are copied onto the 16-byte grid, and results copied back, in one
// launch each.
struct Copies {
  RealignBatch in{}, out{};
  uint8_t* at;
  int sms;
  static int pad(int cols) { return (cols + 7) / 8 * 8; }
  static size_t bytes(int rows, int ld) { return lora_round256(2 * static_cast<size_t>(rows) * ld); }
  uint16_t* take(int rows, int ld) {
    uint16_t* const p = reinterpret_cast<uint16_t*>(at);
    at += bytes(rows, ld);
    return p;
  }
  void add(RealignBatch& b, const uint16_t* src, int lds, uint16_t* dst, int ldd, int rows, int cols,
           int width) {
    const long long blocks = (1ll * rows * (width / 8) + 255) / 256;
    b.job[b.n] = RealignJob{src, lds, dst, ldd, rows, cols, width};
    b.end[b.n] = (b.n ? b.end[b.n - 1] : 0) + static_cast<int>(std::max(1ll, std::min(blocks, 8ll * sms)));
    ++b.n;
  }
  // rows x cols; or two such halves, `up` columns apart in the copy
  void fetch(const uint16_t* src, int lds, uint16_t* dst, int ldd, int rows, int cols, int up = 0) {
    add(in, src, lds, dst, ldd, rows, cols, pad(cols));
    if (up) add(in, src + cols, lds, dst + up, ldd, rows, cols, pad(cols));
  }
  void put(const uint16_t* src, int lds, uint16_t* dst, int ldd, int rows, int cols, int up = 0) {
    add(out, src, lds, dst, ldd, rows, cols, pad(cols) + 16);
    if (up) add(out, src + up, lds, dst + cols, ldd, rows, cols, pad(cols) + 16);
  }
};

// The gradients.  Where whole tiles compute the gate's, matrices off the grid are
// copied here, once for all three products; G's and U's columns then lie a multiple of eight
// apart, with zeros between them in W and dGU, which add nothing to dX.  2000 x 1501 x 2*1111: 71 us
// (1504 x 2*1112, no copies: 51; copied for each product by itself 37 more than here).
int grad(GradArgs p, const LoraDevice& d, cudaStream_t stream) {
  if (narrow_suits(p.M, 2 * p.N, p.K, folds(2, p.act, p.K), d.sms)) return grad_products(p, d, stream);
  auto off = [](const void* m, int ld) { return misaligned({m}, 16) || ld % 8 != 0; };
  const int n8 = Copies::pad(p.N), k8 = Copies::pad(p.K);
  const bool apart = p.N % 8 != 0;
  const bool x = off(p.X, p.ldx), w = apart || off(p.W, p.ldw), c = off(p.dC, p.lddc);
  const bool gu = apart || off(p.dGU, p.lddgu);
  const bool dx = p.dX && (p.K % 8 != 0 || off(p.dX, p.lddx)), dw = p.dW && (apart || off(p.dW, p.lddw));
  if (!(x || w || c || gu || dx || dw)) return grad_products(p, d, stream);
  const size_t bytes = (x ? Copies::bytes(p.M, k8) : 0) + (w ? Copies::bytes(p.K, 2 * n8) : 0) +
                       (c ? Copies::bytes(p.M, n8) : 0) + (gu ? Copies::bytes(p.M, 2 * n8) : 0) +
                       (dx ? Copies::bytes(p.M, k8) : 0) + (dw ? Copies::bytes(p.K, 2 * n8) : 0);
  void* buf = nullptr;
  if (int rc = realigned_scratch(stream, bytes, &buf)) return rc;
  Copies s;
  s.at = static_cast<uint8_t*>(buf);
  s.sms = d.sms;
  const int half = apart ? p.N : 2 * p.N, up = apart ? n8 : 0;   // as copied
  if (x) {
    uint16_t* const m = s.take(p.M, k8);
    s.fetch(p.X, p.ldx, m, k8, p.M, p.K);
    p.X = m;
    p.ldx = k8;
  }
  if (w) {
    uint16_t* const m = s.take(p.K, 2 * n8);
    s.fetch(p.W, p.ldw, m, 2 * n8, p.K, half, up);
    p.W = m;
    p.ldw = 2 * n8;
  }
  if (c) {
    uint16_t* const m = s.take(p.M, n8);
    s.fetch(p.dC, p.lddc, m, n8, p.M, p.N);
    p.dC = m;
    p.lddc = n8;
  }
  if (gu) {
    uint16_t* const m = s.take(p.M, 2 * n8);
    if (apart) {   // zeros where no gradient is written
      s.add(s.in, m, 2 * n8, m + n8 - 8, 2 * n8, p.M, 0, 8);
      s.add(s.in, m, 2 * n8, m + 2 * n8 - 8, 2 * n8, p.M, 0, 8);
    }
    s.put(m, 2 * n8, p.dGU, p.lddgu, p.M, half, up);
    p.dGU = m;
    p.lddgu = 2 * n8;
  }
  if (dx) {
    uint16_t* const m = s.take(p.M, k8);
    s.put(m, k8, p.dX, p.lddx, p.M, p.K);
    p.dX = m;
    p.lddx = k8;
    p.dx_padded = true;
  }
  if (dw) {
    uint16_t* const m = s.take(p.K, 2 * n8);
    if (p.beta != 0.0f) s.fetch(p.dW, p.lddw, m, 2 * n8, p.K, half, up);
    s.put(m, 2 * n8, p.dW, p.lddw, p.K, half, up);
    p.dW = m;
    p.lddw = 2 * n8;
  }
  if (apart) p.up = n8;
  if (s.in.n) {
    s.in.early = true;
    if (launch_realign_f16(s.in, stream) != cudaSuccess) return GEMM_ERR_CUDA;
  }
  if (int rc = grad_products(p, d, stream)) return rc;
  set_last_path("glu_grad.copied");
  if (!s.out.n) return GEMM_OK;
  return launch_unalign_f16(s.out, stream) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

int device(LoraDevice* d) { return query_device(&d->sms, &d->status, &d->wait_limit_ns); }

int trans_entry(int trans_a, int trans_b, const uint16_t* A, const uint16_t* B, void* C, bool f32,
                int M, int N, int K, int lda, int ldb, int ldc, float alpha, float beta,
                cudaStream_t stream) {
  if (M < 0 || N < 0 || K < 0) return GEMM_ERR_DIM;
  if ((trans_a != 0 && trans_a != 1) || (trans_b != 0 && trans_b != 1)) return GEMM_ERR_ARG;
  if (std::max({M, N, K}) > kMaxDim) return GEMM_ERR_ARG;
  if (!trans_a && !trans_b)
    return f32 ? gemm_f16_f32out(A, B, static_cast<float*>(C), M, N, K, lda, ldb, ldc, alpha, beta,
                                 stream)
               : gemm_f16_ld(A, B, static_cast<uint16_t*>(C), M, N, K, lda, ldb, ldc, alpha, beta,
                             stream);
  if (M == 0 || N == 0) {
    set_last_path("noop");
    return GEMM_OK;
  }
  if (ldc < N || (K > 0 && (lda < (trans_a ? M : K) || ldb < (trans_b ? K : N)))) return GEMM_ERR_LD;
  const bool some = K > 0 && alpha != 0.0f;
  if (!C || (some && (!A || !B))) return GEMM_ERR_NULL;
  if (misaligned({A, B}, 2) || misaligned({C}, f32 ? 4 : 2)) return GEMM_ERR_ARG;
  LoraDevice d{};
  if (int rc = device(&d)) return rc;
  std::unique_lock<std::recursive_mutex> call;
  if (int rc = lock_stream(stream, &call)) return rc;
  if (!some) {
    set_last_path("trans.scale");
    if (!f32) return blank(static_cast<uint16_t*>(C), ldc, M, N, beta, d, stream);
    return launch_scale_f32(static_cast<float*>(C), ldc, M, N, beta, 8 * d.sms, stream) == cudaSuccess
               ? GEMM_OK
               : GEMM_ERR_CUDA;
  }
  return transposed(Trans{A, B, C, f32, trans_a != 0, trans_b != 0, M, N, K, lda, ldb, ldc, alpha, beta},
                    false, 0, nullptr, nullptr, d, stream);
}

}  // namespace
}  // namespace gb300

using namespace gb300;

extern "C" {

int gemm_f16_trans(int trans_a, int trans_b, const uint16_t* A, const uint16_t* B, uint16_t* C,
                   int M, int N, int K, int lda, int ldb, int ldc, float alpha, float beta,
                   cudaStream_t stream) {
  return trans_entry(trans_a, trans_b, A, B, C, false, M, N, K, lda, ldb, ldc, alpha, beta, stream);
}

int gemm_f16_trans_f32out(int trans_a, int trans_b, const uint16_t* A, const uint16_t* B, float* C,
                          int M, int N, int K, int lda, int ldb, int ldc, float alpha, float beta,
                          cudaStream_t stream) {
  return trans_entry(trans_a, trans_b, A, B, C, true, M, N, K, lda, ldb, ldc, alpha, beta, stream);
}

int gemm_f16_glu(const uint16_t* X, const uint16_t* W, uint16_t* C, int M, int N, int K, int act,
                 int ldx, int ldw, int ldc, cudaStream_t stream) {
  if (M < 0 || N < 0 || K < 0) return GEMM_ERR_DIM;
  if (!known_act(act) || N > GEMM_GLU_MAX_N || std::max(M, K) > kMaxDim) return GEMM_ERR_ARG;
  if (M == 0 || N == 0) {
    set_last_path("noop");
    return GEMM_OK;
  }
  if (ldc < N || (K > 0 && (ldx < K || ldw < 2 * N))) return GEMM_ERR_LD;
  if (!C || (K > 0 && (!X || !W))) return GEMM_ERR_NULL;
  if (misaligned({X, W, C}, 2)) return GEMM_ERR_ARG;
  LoraDevice d{};
  if (int rc = device(&d)) return rc;
  std::unique_lock<std::recursive_mutex> call;
  if (int rc = lock_stream(stream, &call)) return rc;
  if (K == 0) {
    set_last_path("glu.blank");
    return blank(C, ldc, M, N, 0.0f, d, stream);
  }
  return gated(GluArgs{X, W, M, N, K, ldx, ldw, act, N}, 1, C, ldc, nullptr, 0, d, stream);
}

int gemm_f16_glu_grad(const uint16_t* dC, const uint16_t* X, const uint16_t* W, uint16_t* dGU,
                      uint16_t* dX, uint16_t* dW, int M, int N, int K, int act, int lddc, int ldx,
                      int ldw, int lddgu, int lddx, int lddw, float beta, cudaStream_t stream) {
  if (M < 0 || N < 0 || K < 0) return GEMM_ERR_DIM;
  if (!known_act(act) || N > GEMM_GLU_MAX_N || std::max(M, K) > kMaxDim) return GEMM_ERR_ARG;
  const bool want_gu = M > 0 && N > 0;   // dGU has elements, and every product some
  const bool want_dx = dX && M > 0 && K > 0, want_dw = dW && N > 0 && K > 0;
  if (!want_gu && !want_dx && !want_dw) {
    set_last_path("noop");
    return GEMM_OK;
  }
  const bool some = want_gu && K > 0;
  if ((want_gu && lddgu < 2 * N) || (some && (lddc < N || ldx < K || ldw < 2 * N)) ||
      (want_dx && lddx < K) || (want_dw && lddw < 2 * N))
    return GEMM_ERR_LD;
  if ((want_gu && !dGU) || (some && (!dC || !X || !W))) return GEMM_ERR_NULL;
  if (misaligned({dC, X, W, dGU, dX, dW}, 2)) return GEMM_ERR_ARG;
  LoraDevice d{};
  if (int rc = device(&d)) return rc;
  std::unique_lock<std::recursive_mutex> call;
  if (int rc = lock_stream(stream, &call)) return rc;
  if (!some) {   // no sums: zeros, and dW as beta leaves it
    set_last_path("glu_grad.blank");
    if (want_gu)
      if (int rc = blank(dGU, lddgu, M, 2 * N, 0.0f, d, stream)) return rc;
    if (want_dx)
      if (int rc = blank(dX, lddx, M, K, 0.0f, d, stream)) return rc;
    return want_dw ? blank(dW, lddw, K, 2 * N, beta, d, stream) : GEMM_OK;
  }
  return grad(GradArgs{dC, X, W, dGU, want_dx ? dX : nullptr, want_dw ? dW : nullptr, M, N, K, act,
                       lddc, ldx, ldw, lddgu, lddx, lddw, N, beta},
              d, stream);
}

}  // extern "C"
