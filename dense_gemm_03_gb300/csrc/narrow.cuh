// narrow.cuh -- what the kernels of products with few rows or few tiles share
// (narrow_stream.cu for halves, i8_stream.cu for 8-bit integers): how the work is cut, the
// sums on their way out of tensor memory, and their meeting in a cluster.
#pragma once

#include <algorithm>

#include "stream_finish.cuh"

namespace gb300 {
namespace {

constexpr int kStepK = 128;
constexpr int kSmemMax = 232448;
constexpr int kPartial = -1;
// how an output is finished (cluster form)
enum Finish { kHalf, kFloat, kGate, kGateGrad, kScaled, kScaledGate };
template <int FIN>
constexpr bool paired() {
  return FIN == kGate || FIN == kGateGrad || FIN == kScaledGate;
}

// The product's tiles: blocks of rows x units of 128 columns of W (of a gate in the cluster
// form 64 and the 64 that they gate), each cut into chunks of 128-deep steps.
struct Tiles {
  int M, N, K;                  // rows; columns of W that exist
  int kb, chunks, units, items; // steps, chunks, units, blocks x units x chunks
  int each, more;               // kb / chunks, kb % chunks
  int unit_cols;                // first columns of units apart
  int rows;                     // rows of a block (at most)
  int n_cols, acc_cols;         // columns of the accumulator
  bool reread;                  // several blocks of rows read W
  bool beside;                  // waits for the kernel before it at the end
  bool vec;                     // results' rows (and dC's) on the grid of four elements
  float* part;
  unsigned long long wait_limit_ns;
  DeviceStatus* status;

  // the first kb % chunks chunks of an output are a step longer than the rest
  __device__ int first_step(int it) const {
    const int c = it % chunks;
    return c * each + min(c, more);
  }
  __device__ int steps(int it) const { return each + (it % chunks < more ? 1 : 0); }
  __device__ int n0(int it) const { return it / chunks % units * unit_cols; }
  __device__ int row0(int it) const { return it / chunks / units * rows; }
};

// Whether the phase is complete, without a pause (try_wait may suspend the thread).
__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}

// The accumulator, 32 columns of W (lanes of this warp's quadrant) by rows of X, to
// out[row][128]; `part` of `parts` warps of the quadrant.  more != 0: the second half of
// the sums lies that many columns on.
__device__ __forceinline__ void write_sums(uint32_t tmem, uint32_t more, int quad, int lane, int part, int parts,
                                           int rows, float* out) {
  const uint32_t d0 = tmem + (static_cast<uint32_t>(32 * quad) << 16);
  out += 32 * quad + lane;
  for (int r0 = 16 * part; r0 < rows; r0 += 16 * parts) {   // n_cols is a multiple of 16
    uint32_t g[8], h[8];
    tmem_ld_32x32b_x8(d0 + r0, g);
    tmem_ld_32x32b_x8(d0 + r0 + 8, h);
    tmem_wait_ld2(g, h);
    if (more) {
      uint32_t a[8], b[8];
      tmem_ld_32x32b_x8(d0 + more + r0, a);
      tmem_ld_32x32b_x8(d0 + more + r0 + 8, b);
      tmem_wait_ld2(a, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        g[i] = __float_as_uint(__uint_as_float(g[i]) + __uint_as_float(a[i]));
        h[i] = __float_as_uint(__uint_as_float(h[i]) + __uint_as_float(b[i]));
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (r0 + i < rows) out[(r0 + i) * 128] = __uint_as_float(g[i]);
      if (r0 + 8 + i < rows) out[(r0 + 8 + i) * 128] = __uint_as_float(h[i]);
    }
  }
}

// Cluster form, all threads of all its CTAs: every chunk's sums lie at `sums` in its
// CTA's shared memory; each CTA adds up and finishes its share of the tile's outputs.
template <int FIN>
__device__ __forceinline__ void cluster_finish(const Tiles& p, const StreamSum& fin, uint32_t sums,
                                               int threads) {
  __syncwarp();
  // every chunk's sums are there
  if (p.chunks > 1)
    cluster_sync();
  else
    __syncthreads();
  constexpr int kGateOf = FIN == kGateGrad ? 2 : (paired<FIN>() ? 1 : 0);
  constexpr int kQuads = paired<FIN>() ? 16 : 32;   // quads of output columns in a unit
  const int it = blockIdx.x, rank = it % p.chunks, row0 = p.row0(it);
  const int total = min(p.rows, p.M - row0) * kQuads;
  for (int i = rank * total / p.chunks + static_cast<int>(threadIdx.x);
       i < (rank + 1) * total / p.chunks; i += threads) {
    const int r = i / kQuads, q = i % kQuads;
    const int c = p.n0(it) + 4 * q, n = min(4, fin.N - c);
    if (n <= 0) continue;
    const uint32_t at = sums + static_cast<uint32_t>((r * 128 + 4 * q) * 4);
    float s[4] = {}, u[4] = {};
    auto add = [](float (&a)[4], float4 v) {
      a[0] += v.x;
      a[1] += v.y;
      a[2] += v.z;
      a[3] += v.w;
    };
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < p.chunks) {
        const uint32_t peer = map_to_cta(at, j);
        add(s, ld_cluster_f4(peer));
        if (paired<FIN>()) add(u, ld_cluster_f4(peer + 256));
      }
    stream_finish<kGateOf, FIN == kFloat, FIN == kScaled || FIN == kScaledGate, 4>(
        fin, row0 + r, c, n, p.vec && n == 4, s, u);
  }
  if (p.chunks > 1) cluster_sync();   // nobody leaves while its sums are being read
  else __syncthreads();
}

// ------------------------------------------------------------------- plans
// The cluster form's chunks for `tiles` tiles of `steps` steps: as many as one wave of
// CTAs leaves room for (76, 36 and 15 clusters of 2, 4 and 8 CTAs fit on 152 SMs); 0: it
// does not suit.
inline int cluster_chunks(long long tiles, int steps, int sms) {
  if (tiles > sms) return 0;
  int best = 1;
  for (int c = 2; c <= 8; c *= 2)
    if (tiles * c <= (c <= 2 ? sms : c == 4 ? sms - 8 : sms - 32) && steps >= c) best = c;
  return best;
}

// Whether the cluster form is expected to be faster than partial sums over all SMs: these
// share the steps out evenly but take 3.3 us more (a second kernel, sums through L2).  A
// step takes about 0.3 us and 0.003 for each row of the block.  (8 tiles of 256 x 128 over
// 64 steps, 64 CTAs: cluster 13.9 us, partial 12.2.)
inline bool cluster_pays(const Tiles& a, int sms) {
  if (a.chunks == 0) return false;
  const double longest = (a.kb + a.chunks - 1) / a.chunks;
  const double even = 1.0 * a.items / a.chunks * a.kb / sms;
  return (longest - even) * (0.3 + 0.003 * a.n_cols) < 3.3;
}

inline void common_tiles(Tiles& a, int M, int K, int rows, bool trans_x, const LoraDevice& d) {
  a.M = M;
  a.K = K;
  a.rows = block_rows(M, rows, trans_x);
  a.kb = (K + kStepK - 1) / kStepK;
  a.n_cols = (a.rows + 15) / 16 * 16;
  a.acc_cols = 32;
  while (a.acc_cols < a.n_cols) a.acc_cols *= 2;
  a.reread = M > rows;
  a.wait_limit_ns = d.wait_limit_ns;
  a.status = d.status;
}

inline void cut(Tiles& a, long long tiles, int chunks) {
  a.chunks = chunks;
  a.each = chunks ? a.kb / chunks : 0;
  a.more = a.kb - a.each * chunks;
  a.items = static_cast<int>(tiles * chunks);
}

// Partial sums over persistent CTAs.
inline Tiles partial_tiles(int M, int cols, int K, int rows, bool trans_x, int kb16, int least,
                           const LoraDevice& d) {
  Tiles a{};
  common_tiles(a, M, K, rows, trans_x, d);
  const int blocks = (M + a.rows - 1) / a.rows;
  a.N = cols;
  a.units = (cols + 127) / 128;
  a.unit_cols = 128;
  cut(a, 1ll * blocks * a.units,
      std::min(a.kb, plan_chunks(a.units, blocks, kb16, a.rows, d.sms, least)));
  return a;
}

// The cluster form; chunks == 0: it does not suit.
inline Tiles cluster_tiles(const StreamSum& s, int K, int rows, bool trans_x, const LoraDevice& d) {
  Tiles a{};
  common_tiles(a, s.M, K, rows, trans_x, d);
  const int blocks = (s.M + a.rows - 1) / a.rows;
  a.N = s.gate ? 2 * s.N : s.N;
  a.unit_cols = s.gate ? 64 : 128;
  a.units = (s.N + a.unit_cols - 1) / a.unit_cols;
  const long long tiles = 1ll * blocks * a.units;
  cut(a, tiles, cluster_chunks(tiles, a.kb, d.sms));
  uintptr_t bits = reinterpret_cast<uintptr_t>(s.C);
  a.vec = s.ldc % 4 == 0;
  if (s.gate == 2) {
    bits |= reinterpret_cast<uintptr_t>(s.g.dC) | reinterpret_cast<uintptr_t>(s.g.dU);
    a.vec = a.vec && s.g.lddc % 4 == 0;
  }
  a.vec = a.vec && bits % (s.f32 ? 16 : 8) == 0;
  return a;
}

// A launch of `grid` CTAs, in clusters of `chunks` (0: none).  CTAs of a cluster wait for one
// another, and for tensor memory that a CTA beside them on the SM may hold: two clusters
// with a CTA each on the same two SMs could wait for ever.  So they take all of an SM's
// shared memory, and no other CTA that uses tensor memory (which all use shared memory)
// is there beside them.
template <class K, class... A>
int launch_narrow(K kernel, int threads, size_t smem, int grid, int chunks, bool* configured,
                  cudaStream_t stream, const A&... args) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return GEMM_ERR_CUDA;
  if (dev < 64 && !configured[dev]) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax) !=
        cudaSuccess)
      return GEMM_ERR_CUDA;
    configured[dev] = true;
  }
  cudaLaunchAttribute attr[2];
  unsigned int n = 0;
  if (chunks) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = static_cast<unsigned>(chunks);
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // see launch_early
  attr[n].val.programmaticStreamSerializationAllowed = 1;
  ++n;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = chunks > 1 ? kSmemMax : smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return counted_launch(cudaLaunchKernelEx(&cfg, kernel, args...)) == cudaSuccess ? GEMM_OK
                                                                                  : GEMM_ERR_CUDA;
}

}  // namespace
}  // namespace gb300
