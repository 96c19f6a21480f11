// internal.h -- declarations shared by the host dispatcher and the kernel
// translation units.  Not part of the public ABI.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>
#include <mutex>

namespace gb300 {

// Every kernel launch of the library goes through counted_launch: a
// successful launch adds one to a process-wide counter (gemm_launch_count).
void note_launch();
// Records the path the current call on this thread takes (a static string);
// gemm_last_path() returns it.
void set_last_path(const char* path);
inline cudaError_t counted_launch(cudaError_t e) {
  if (e == cudaSuccess) note_launch();
  return e;
}

struct DeviceStatus;

// Operand-load modes of the tensor-core kernel.
enum LoadMode : int { kLoadTma = 0, kLoadManual = 1 };
// Epilogue modes: TMA load/store of C, predicated element access of C, or
// raw fp32 partial sums to the split-K workspace.
// kEpiF32: fp32 C from registers; kEpiF32Tma: fp32 C through shared memory
// and TMA (CTA pairs, C 16-byte aligned, N % 4 == 0).
enum EpiMode : int { kEpiTma = 0, kEpiManual = 1, kEpiPartial = 2, kEpiF32 = 3, kEpiF32Tma = 4 };

// Division of numbers below 2^32 by a fixed one, as a multiplication.
struct FastDiv {
  unsigned long long m;   // 2^64 / d rounded up (0: d is 1)
  unsigned int d;
#ifdef __CUDACC__
  __device__ int div(int n) const {
    return m ? static_cast<int>(__umul64hi(m, static_cast<unsigned int>(n))) : n;
  }
#endif
};
inline FastDiv fast_div(long long d) {
  return FastDiv{d > 1 ? ~0ull / static_cast<unsigned long long>(d) + 1 : 0,
                 static_cast<unsigned int>(d)};
}

struct TcArgs {
  const uint16_t* A;
  const uint16_t* B;
  uint16_t* C;
  int M, N, K;
  long long lda, ldb, ldc;
  float alpha, beta;
  int tiles_m, tiles_n;
  int splits;         // number of K slices (1 = no split)
  int kb_total;       // ceil(K / 64)
  int kb_per_split;   // K blocks per slice (every slice non-empty)
  int num_units;      // dp_tiles * splits + tail tiles * tail_splits
  int group_m;        // tile-order grouping along M (L2 reuse of B panels)
  // by group_m * tiles_n, group_m, and the tile rows of the last group: a thread's
  // divisions took 0.6 us before its first load (set_divisors)
  FastDiv by_group, by_gm, by_last;
  void set_divisors() {
    by_group = fast_div(1ll * group_m * tiles_n);
    by_gm = fast_div(group_m);
    by_last = fast_div((tiles_m - 1) % group_m + 1);
  }
  float* ws;          // split-K partials [splits][M][ws_ld]
  long long ws_ld;
  // Tail balancing (splits == 1 only): the first dp_tiles tiles (in visiting
  // order) are computed whole; each remaining tile is cut into tail_splits
  // K slices whose fp32 partial sums go to tail_ws; the last slice to finish
  // (counted in tail_counters under this launch's epoch) adds them up in
  // slice order and runs the epilogue.
  int dp_tiles;
  int tail_splits;
  int tail_kb_per_split;
  float* tail_ws;                      // [tail tile][slice][128][BN]
  unsigned long long* tail_counters;   // [tail tile][8 epilogue warps]: epoch << 32 | arrivals
  unsigned int epoch;
  // Stream-K region (sk_tiles > 0, after the units above): the tiles
  // sk_tile0 .. sk_tile0 + sk_tiles - 1 (in visiting order) are treated as
  // sk_iters = sk_tiles * kb_total k-blocks, and worker w of sk_workers takes
  // k-blocks [w*sk_iters/sk_workers, (w+1)*sk_iters/sk_workers), cut at tile
  // boundaries into pieces.  A tile covered by several pieces is finished like
  // a tail tile; tail_splits is then the most pieces any tile can have (the
  // stride of tail_ws).
  int sk_tile0, sk_tiles, sk_workers;
  long long sk_iters;
  // sk_order 0: a worker takes its stream-K pieces after its whole tiles, in
  // k order.  sk_order 1 (the stream-K tiles are the last, partial wave and no
  // range is longer than a tile, so a range touches at most two tiles): the
  // piece that ends a tile (it finishes the tile) runs last, after the whole
  // tiles, and the other piece runs first, so that a tile's other pieces have
  // long published when its finisher ends.
  int sk_order;
  // kEpiF32: C is fp32 (Cf, ldc in floats) and written straight from
  // registers, with 16-byte accesses when vec_c (Cf and ldc 16-byte aligned)
  // and predicated element accesses otherwise.
  float* Cf;
  int vec_c;
  // tail_halves != 0 (TMA loads, BN >= 128): the tiles after dp_tiles are
  // computed as two units of BN/2 columns each (whole K, an MMA of N = BN/2)
  // instead of K slices.
  int tail_halves;
  // tail_first != 0 (splits == 1, tail_splits == 2, K slices of
  // tail_kb_per_split k-blocks and the rest): the first T tiles in visiting
  // order are cut in two; units [0, T) are their first K slices, then come the
  // dp_tiles whole tiles T, T + 1, ..., then the second slices.  Workers take
  // units worker, worker + nworkers, ..., so a first slice (it publishes its
  // partial sums) is its worker's first unit and a second slice (it finishes
  // the tile) its worker's last, long after the first was published.
  int tail_first;
  // single-CTA kernels: A (B) is read by one column (row) of tiles only, i.e.
  // streamed once -- loaded evict-first, so it does not push out of L2 lines
  // that are still useful (or dirty lines that would be written back)
  int stream_a, stream_b;
  // adapters: A, B or C was copied by the kernel launched just before
  int wait_operands;
  // started beside the kernel before it, on operands that one waited for: waits at its end
  int beside;
  unsigned long long wait_limit_ns;
  DeviceStatus* status;
  // host only: may start early (programmatic dependent launch: the kernel waits for
  // the one before it on the stream before it touches global memory), as a kernel
  // that follows this call's pre-pass does
  bool pdl;
};

// Low-rank adapters picked by row beside a GEMM on CTA pairs (256-row tiles):
// what the kernel needs beside the product's own operands.
constexpr int kLoraListStride = 257;   // a 256-row block's list: count, adapters
constexpr int kLoraBadParts = 4;
struct LoraTailArgs {
  const float* V;        // [M][ldv] fp32, the rows' low-rank products
  const uint16_t* packed;   // the same as halves, [M][chunk][32 hi, 32 lo]
  const uint8_t* apart;     // [M] 1: past the half range, packed is zero and V added in
                            // fp32; 2: what packed leaves out is, where weights are large
  int ldv;
  const int* ids;        // [M]
  const int* lists;      // [256-row block][kLoraListStride]: its distinct adapters
  const int* bad;        // [adapters][kLoraBadParts], of the weights of that part of F[a]:
                         // 1 when some are not finite, 2 when some are large
  const uint16_t* F;     // the adapters' B operand (for the bad ones)
  long long ldf, f_stride;
  int R, adapters, chunks;   // chunks of 32 ranks
};
// A call of the pair kernel with adapters: `trans` when B is stored N x K and
// F[a] N x R (the gradient with respect to the left operand).
struct LoraCall {
  LoraTailArgs tail;
  bool trans;
};
// C := alpha (A B + V F) + beta C through the pair kernel, after the
// kernels on `stream` that write V, the lists and the marks.  F has rows on the
// 16-byte grid.  Returns a GEMM_* code.
int gemm_f16_lora_pair(const uint16_t* A, const uint16_t* B, uint16_t* C, int M, int N, int K,
                       long long lda, long long ldb, long long ldc, float alpha, float beta,
                       const LoraCall& lora, cudaStream_t stream);
cudaError_t launch_gemm_f16_tc_lora(bool trans, int epi_mode, const CUtensorMap& tmA,
                                    const CUtensorMap& tmB, const CUtensorMap& tmC,
                                    const CUtensorMap& tmE, const CUtensorMap& tmV,
                                    const LoraTailArgs& tail,
                                    const TcArgs& args, int grid, cudaStream_t stream);

// What a gated or scaled product needs beside the product's own operands.
struct GateArgs {
  int act;             // GEMM_ACT_*
  int up;              // columns of B from a gate's to the one it gates
  const uint16_t* dC;  // gradient: M x N, rows lddc apart
  long long lddc;
  uint16_t* dU;        // gradient: beside C (dG), the same leading dimension
  const float *sx, *sw;   // scales by row and by column of B (NULL: ones)
};
// Variants of the pair kernel: operands stored transposed (half or float C) ...
cudaError_t launch_gemm_f16_tc_trans(bool trans_a, bool trans_b, int epi_mode,
                                     const CUtensorMap& tmA, const CUtensorMap& tmB,
                                     const CUtensorMap& tmC, const TcArgs& args, int grid,
                                     cudaStream_t stream);
// ... gated products (gate 1), their gradient (gate 2), and products scaled by row and
// column (gate 0 or 1); tmU: dU's map (gate 2); fold: G and U folded (gate 2, see the kernel).
cudaError_t launch_gemm_f16_tc_gate(int gate, bool scaled, bool fold, int epi_mode, const CUtensorMap& tmA,
                                    const CUtensorMap& tmB, const CUtensorMap& tmC,
                                    const CUtensorMap& tmU, const GateArgs& gate_args,
                                    const TcArgs& args, int grid, cudaStream_t stream);
// A product through one of those variants.  op(A) is M x K, op(B) K x N; with
// `gate` B is K x (up + N) and C the gated result (gate 1), or dG with dU beside it
// (gate 2).  C is float when c_f32.  Rows of A and B, and of a half C, that are off
// the 16-byte grid are copied.  Returns a GEMM_* code.
//
// Two products of one call whose operands the kernel before both wrote can run side
// by side: the second names what the first left behind (`before`).  A pair kernel lets the kernel
// after it start only when it has itself waited for the one before, so what it reads is
// there for the second too, which waits for the first only as it ends (the order on the
// stream then holds for all that follows).  The second must not need a copy of an operand,
// which another kernel would make, nor scratch that the first uses.
struct PairDone {
  bool pair;       // the last kernel is a pair kernel
  bool parts;      // that keeps partial sums in scratch
};
struct PairCall {
  const uint16_t *A, *B;
  void* C;
  bool c_f32;
  int M, N, K;
  long long lda, ldb, ldc;
  float alpha, beta;
  bool trans_a, trans_b;
  int gate;
  bool scaled;
  bool fold;               // gate 2: long sums folded into registers
  GateArgs g;
  bool c_padded;           // C's columns up to a multiple of eight may be written
  bool whole;              // no half-width tiles: they would take SMs of a product beside
  int pairs;               // of SMs at most (0: all)
  const PairDone* before;  // see above; or NULL
  PairDone* done;          // or NULL
};
int gemm_f16_pair(const PairCall& call, cudaStream_t stream);

// Tensor-core fp16 GEMM (tcgen05).  Maps are ignored by the modes that do not
// use them.  kpb: k-blocks per ring stage, 1, or 2 for 64-wide tiles with TMA
// loads and epilogue.  Returns a cudaError_t from the launch.
cudaError_t launch_gemm_f16_tc(int bn, int load_mode, int epi_mode, const CUtensorMap& tmA,
                               const CUtensorMap& tmB, const CUtensorMap& tmC, const TcArgs& args,
                               int grid, cudaStream_t stream, int kpb = 1);
int tc_threads(int load_mode);

// The same GEMM with an fp32 C (epilogue kEpiF32; gemm_f16_f32out.cu).
cudaError_t launch_gemm_f16_tc_f32(int bn, int load_mode, const CUtensorMap& tmA,
                                   const CUtensorMap& tmB, const TcArgs& args, int grid,
                                   cudaStream_t stream);
cudaError_t launch_gemm_f16_tc_pair_f32(int epi_mode, const CUtensorMap& tmA,
                                        const CUtensorMap& tmB, const CUtensorMap& tmC,
                                        const TcArgs& args, int grid, cudaStream_t stream);
int tc_pair_max_clusters_f32(int epi_mode);

// The same GEMM (128-wide tiles, TMA loads, one CTA per tile) for M <= am,
// staging am = 32 or 64 rows of A per k-block (gemm_f16_skinny.cu).
cudaError_t launch_gemm_f16_tc_skinny(int am, int epi_mode, const CUtensorMap& tmA,
                                      const CUtensorMap& tmB, const CUtensorMap& tmC,
                                      const TcArgs& args, int grid, cudaStream_t stream);
// 64-wide tiles of 64 rows (tcgen05.mma with M = 64), TMA loads and epilogue,
// whole-K units only (gemm_f16_skinny.cu); C's map has 32 x 16-row boxes.
cudaError_t launch_gemm_f16_tc_m64(const CUtensorMap& tmA, const CUtensorMap& tmB,
                                   const CUtensorMap& tmC, const TcArgs& args, int grid,
                                   cudaStream_t stream);

// One thread waits on an mbarrier that nothing arrives on, so the bounded wait
// runs out after limit_ns and records GEMM_ERR_TIMEOUT in *status.
cudaError_t launch_wait_probe(unsigned long long limit_ns, DeviceStatus* status,
                              cudaStream_t stream);

// fp32 -> fp16 conversion of n elements, round to nearest even.
cudaError_t launch_f32_to_f16(const float* src, uint16_t* dst, long long n, int grid,
                              cudaStream_t stream);

// The same GEMM on CTA pairs (clusters of 2 sharing tcgen05.mma.cta_group::2):
// 256 x bn output tiles (bn = 256, or 224 / 192 with a half C), TMA operand
// loads only, epilogue kEpiTma or kEpiManual (or the fp32-C ones, bn = 256).
// tiles_m counts 256-row tiles; grid = 2 x (number of pairs).  kpb: k-blocks
// per ring stage, 1, or 2 for bn = 256 with the TMA epilogue.
cudaError_t launch_gemm_f16_tc_pair(int bn, int epi_mode, const CUtensorMap& tmA,
                                    const CUtensorMap& tmB, const CUtensorMap& tmC,
                                    const TcArgs& args, int grid, cudaStream_t stream,
                                    int kpb = 1);
// The 224- and 192-wide instances (gemm_f16_pair_narrow.cu).
cudaError_t launch_gemm_f16_tc_pair_narrow(int bn, int epi_mode, const CUtensorMap& tmA,
                                           const CUtensorMap& tmB, const CUtensorMap& tmC,
                                           const TcArgs& args, int grid, cudaStream_t stream);
// Pairs of the 256-wide configuration that fit on the device at once (0 on
// error); the narrower tiles stage the same bytes, so the same number fits.
int tc_pair_max_clusters(int epi_mode);

// Split-K reduction: C = half(alpha * sum_s ws[s] + beta * C).
cudaError_t launch_splitk_reduce_f16(const float* ws, long long ws_ld, int splits, uint16_t* C,
                                     long long ldc, int M, int N, float alpha, float beta,
                                     int grid, cudaStream_t stream);

// A launch that may begin while the kernel before it on the stream, whoever
// launched that, is in its last blocks, so that its own set-up is not waited for.  The kernel
// waits (griddep_wait) for all of that one before it touches global memory, and so for
// everything before that: the stream's order is as without.  Calls back to back, on a
// GB300: one token of 2048 x 2*4096 in halves 11.0 -> 9.3 us, one of 4096 x 4096 in 8
// bits 11.6 -> 9.2, 331 x 2048 x 4096 14.4 -> 12.1.
template <class K, class... A>
cudaError_t launch_early(K kernel, unsigned grid, unsigned threads, size_t smem, cudaStream_t stream,
                         const A&... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Copies a rows x cols half matrix with any leading dimension and alignment
// into a 16-byte-aligned one with ldd = cols rounded up to 8 (zero padding), or
// into `width` columns (a multiple of 8, at least cols) of one with a larger ldd.
struct RealignJob {
  const uint16_t* src;
  long long lds;
  uint16_t* dst;
  long long ldd;
  int rows, cols;
  long long width = 0;   // 0: ldd
};
// One launch for several copies: blocks [end[i-1], end[i]) copy jobs[i].
constexpr int kRealignJobs = 8;
struct RealignBatch {
  RealignJob job[kRealignJobs];
  int end[kRealignJobs];
  int n;
  bool early = false;   // see launch_early
};
cudaError_t launch_realign_f16(const RealignBatch& batch, cudaStream_t stream);

// The copies back: dst (rows x cols, any 2-byte alignment and leading dimension
// ldd) := src (16-byte-aligned rows, lds >= cols rounded up to 8).  Launched
// after the kernel that writes src, which it may overlap (programmatic
// dependent launch; it waits for that kernel's completion before reading).
cudaError_t launch_unalign_f16(const RealignBatch& batch, cudaStream_t stream);

// Both splits of a 3xTF32 product in one launch: A (M x K) into Ab, As and
// B^T (B is K x N) into Bb, Bs, all with leading dimension ld2 (>= K, % 4 == 0);
// grid_a blocks work on A, grid_b on B^T.
cudaError_t launch_split_tf32_ab(const float* A, long long lda, float* Ab, float* As,
                                 const float* B, long long ldb, float* Bb, float* Bs, long long ld2,
                                 int M, int N, int K, int grid_a, int grid_b, cudaStream_t stream);

// The fp16 parts of the 3xFP16 SGEMM, x * 2^e = h1 + h2 (+ 2^-22 relative):
// 3xFP16 operand parts: A1, A2 (M x lda2 halves) and B1, B2 (K x ldb2), and
// the power-of-two exponents they were scaled by, per K chunk of
// kF16x3ChunkK: ea[row][chunk] (M x kchunks), eb[chunk][col] (kchunks x ldeb,
// ldeb >= N + 4).
constexpr int kF16x3ChunkK = 256;
struct F16x3Parts {
  uint16_t *A1, *A2, *B1, *B2;
  long long lda2, ldb2;
  int* ea;
  int* eb;
  long long ldeb;
};
// One launch of 1024-thread blocks: blocks [0, grid_b) split B by (chunk,
// 128 columns), the other grid_a blocks A by (row, chunk), one warp an item.
cudaError_t launch_f16x3_split(const float* A, long long lda, const float* B, long long ldb,
                               const F16x3Parts& parts, int M, int N, int K, int grid_a,
                               int grid_b, cudaStream_t stream);

// 3xTF32 SGEMM on CTA pairs: C = alpha*(Ab*Bb + Ab*Bs + As*Bb) + beta*C with
// the split operands dense and K-contiguous: A parts M x roundup(K,4), B parts
// transposed, N x roundup(K,4).
// k-blocks (64 bytes of K per row) in one TMEM accumulation chunk of the
// split-operand kernel: 128 floats (3xTF32) or 256 halves (3xFP16).
constexpr int kSplitChunkKb = 8;
struct Tf32Args {
  const float* Ab;
  const float* As;
  const float* Bb;
  const float* Bs;
  float* C;
  int M, N, K;
  long long ldc;
  float alpha, beta;
  int tiles_m, tiles_n;   // 256 x 256 pair tiles
  int kb_total;           // ceil(K / 32)
  // units [0, dp_tiles) are whole tiles; each tile after them (the last,
  // partial wave) runs as two half-width units of 128 columns
  int dp_tiles;
  int num_units;
  int group_m;
  bool vec_c;             // C 16-byte aligned with ldc % 4 == 0
  unsigned long long wait_limit_ns;
  DeviceStatus* status;
  // splits > 1: every unit is one K slice of a whole tile (unit = tile *
  // splits + slice, slice s covering k-blocks [s * kb_per_split, ...), a
  // multiple of the 4-k-block accumulation chunk); each slice publishes fp32
  // partial sums and the last one of a tile to finish adds them up in slice
  // order and writes C
  int splits;
  int kb_per_split;
  float4* part_ws;                  // [tile][rank][warp][slice][32 column quads][32 rows]
  unsigned long long* counters;     // [tile][rank][warp]: (epoch << 32) | arrivals
  unsigned int epoch;
  bool pdl;                         // host only: as TcArgs::pdl (after the split pre-pass)
  // Two-slice tail (splits == 1): the tail tiles -- T = (num_units -
  // dp_tiles) / 2 of them, the first T in visiting order -- are cut into a
  // first slice of kb_per_split k-blocks (whole accumulation chunks), a
  // worker's first unit, and a second slice, a worker's last; the slice that
  // arrives last adds both up, as with K slices.
  int tail_first;
  // 3xFP16 only: the power-of-two exponents the parts were scaled by, per K
  // chunk of kF16x3ChunkK (the accumulation chunk): ea[row * kchunks + c],
  // eb[c * ldeb + col] (ldeb >= N + 4)
  const int* ea;
  const int* eb;
  long long ldeb;
  int kchunks;
};
// tmBbh / tmBsh: the B parts with 64-row boxes, for the half-width units.
cudaError_t launch_sgemm_3xtf32(const CUtensorMap& tmAb, const CUtensorMap& tmAs,
                                const CUtensorMap& tmBb, const CUtensorMap& tmBs,
                                const CUtensorMap& tmBbh, const CUtensorMap& tmBsh,
                                const Tf32Args& args, int grid, cudaStream_t stream);
int sgemm_3xtf32_max_pairs();
// The same kernel on the 3xFP16 parts (A1, A2: M x lda2 halves, boxes of 64
// columns x 128 rows; B1, B2: K x ldb2 halves, boxes of 64 columns x 64 rows);
// k-blocks of 64.
cudaError_t launch_sgemm_3xf16(const CUtensorMap& tmA1, const CUtensorMap& tmA2,
                               const CUtensorMap& tmB1, const CUtensorMap& tmB2,
                               const Tf32Args& args, int grid, cudaStream_t stream);

// C := beta * C (C := 0 when beta == 0): the alpha == 0 / K == 0 case.
cudaError_t launch_scale_f16(uint16_t* C, long long ldc, int M, int N, float beta, int grid,
                             cudaStream_t stream);
cudaError_t launch_scale_f32(float* C, long long ldc, int M, int N, float beta, int grid,
                             cudaStream_t stream);

// FFMA SGEMM.  vec = 16-byte vector loads allowed (aligned pointers, ld % 4 == 0).
struct SgemmArgs {
  const float* A;
  const float* B;
  float* C;
  int M, N, K;
  long long lda, ldb, ldc;
  float alpha, beta;
};
cudaError_t launch_sgemm_ffma(bool vec, const SgemmArgs& args, cudaStream_t stream);

// Current device: SM count, status word and wait limit (library set-up done
// on first use).  Returns a GEMM_* code.
int query_device(int* sm_count, DeviceStatus** status, unsigned long long* wait_limit_ns);

// To be held from the first routed_scratch() of a call to its last launch.
// Returns a GEMM_* code.
int lock_stream(cudaStream_t stream, std::unique_lock<std::recursive_mutex>* call);

// Scratch of the row-routed products (adapters, experts) on `stream`, at least
// `bytes` long and 256-byte aligned; kept per device and stream, freed by
// gemm_release().  Returns a GEMM_* code.
// `zeroed`: a separate region of at least that many bytes that starts at zero
// when it is first handed out and then keeps what kernels leave in it.
int routed_scratch(cudaStream_t stream, size_t bytes, void** out, size_t zeroed = 0,
                   void** zeroed_out = nullptr);
// The buffer of the copies that gemm_f16_pair makes (it makes none of operands on the grid).
int realigned_scratch(cudaStream_t stream, size_t bytes, void** out);
// Tensor map of a stack of `depth` fp16 matrices (rows x cols, leading
// dimension ld, `stride` elements apart), 128-, 64- or 32-byte swizzle, boxes of
// box_cols x box_rows of one matrix; what lies outside a matrix reads as zero.
int encode_map_f16_stack(CUtensorMap* map, const void* ptr, int rows, int cols, long long ld,
                         int depth, long long stride, int box_cols, int box_rows,
                         int swizzle = 128);

// 2-D fp16 tensor map with 128-byte swizzle (rows x cols, row stride ld).
int encode_map_f16(CUtensorMap* map, const void* ptr, int rows, int cols, long long ld,
                   int box_cols, int box_rows);
// Map of two dimensions (the third's size 0) or three over elements of `elem` bytes (1: bytes, 2:
// halves): sizes, the strides of the second and third dimension in elements, and the box;
// its rows are 64 or 128 bytes, swizzled over that width.
struct MapDims {
  long long d[3];
};
int encode_map_3d(CUtensorMap* map, int elem, const void* ptr, MapDims size, MapDims stride,
                  MapDims box);

}  // namespace gb300
