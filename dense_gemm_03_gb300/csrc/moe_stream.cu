// moe_stream.cu -- the mixture-of-experts layer for a few tokens in two
// kernels that read each chosen expert's weights once.
//
//   moe_logits_kernel  l = x Wr as K slices over many CTAs; the CTA that ends a
//                      block of four tokens adds the slices up in order, picks
//                      the topk experts and writes ids and p.
//   moe_stream_kernel  one CTA per SM:
//     up    hid = silu(x W1g) .* (x W1u) of every (token, expert) pair
//     down  z = hid W2 per pair
//     sum   y = sum_k p_k z_k + beta y
//
// With n tokens at an expert a weight takes part in n multiply-adds, far fewer
// than the ~280 per byte at which the tensor cores bind: the time is that of
// streaming the weights from HBM.  So the weights are the M operand: a unit is
// 128 + 128 columns of an expert's matrix (gate and up columns j, or 256
// columns of W2) in two TMEM accumulators, the expert's tokens the N operand
// (N = 16..128), and a k-block is 64 rows of the matrix, 32 KB by TMA.
//
// Units are cut along K into chunks of equal length, numbered up first, and
// CTAs take chunk numbers from a counter, in order: SMs stream at rates up to
// 20% apart, and an equal share for each left the fast ones idle.  A unit's chunks publish fp32
// partial sums; the last chunk of an up unit to arrive adds them in k order
// (so the result does not depend on which that is), the sum step does so for
// down units.  A down chunk waits until its own expert's hid is written, the
// sum step for all down chunks; both wait only for chunks of lower numbers,
// which running CTAs have taken and finish without waiting for later ones, so
// no wait needs a CTA that has not started.  The weights do not depend on those
// waits: W2 streams into the ring across them.
//
// hid is fp32.  For the second product each pair's row is scaled by the power of
// two that brings its largest finite magnitude into [2^13, 2^14) and staged as two
// halves, hi + lo (22 significant bits or 2^-37 of the largest), separate rows of
// the N operand whose products are added up and scaled back after it: the layer's
// only rounding to half is that of Y, and a gated row of any size has its bits.  A
// token's columns never mix with another's, and a pair's partial results are read
// only for its own token.
//
// Shared memory per ring stage: four 64-column boxes of 64 k-rows (128-byte
// swizzle, MN-major: LBO 8 KB to the next 64 columns, SBO 1 KB to the next 8
// k-rows), then the token rows, 128 bytes of k each (K-major, SBO 1 KB).
#include <algorithm>
#include <cstddef>

#include "gemm.h"
#include "moe.h"

namespace gb300 {
namespace {

constexpr int kBlockT = 64;                  // most tokens per launch

// ------------------------------------------------------------------ routing
constexpr int kRouteThreads = 256;
constexpr int kRouteWarps = kRouteThreads / 32;
constexpr int kRouteT = 4;                   // tokens per CTA
constexpr int kMaxSplits = 16;
constexpr int kRouteChunk = 512;             // rows of Wr staged against at a time

struct RouteArgs {
  const uint16_t *X, *Wr;
  long long ldx;
  int T, H, E, topk, renormalize;
  int egroups, tblocks, splits, rows_per_split;
  float* part;             // [split][T][E]
  unsigned int* counters;  // [tblock]; zero between launches
  int* ids;                // [T][topk] for moe_stream_kernel, and the caller's
  float* probs;
  int* ids_out;
  float* probs_out;
  // words that moe_stream_kernel needs at zero
  unsigned int* zero;
  int nzero;
};

__global__ void __launch_bounds__(kRouteThreads) moe_logits_kernel(const RouteArgs a) {
  __shared__ float xs[kRouteT][kRouteChunk];
  __shared__ float part[kRouteWarps][kRouteT][32];
  __shared__ int last;
  extern __shared__ float logits[];          // [kRouteT][E]
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = blockIdx.x * kRouteThreads + threadIdx.x; i < a.nzero;
       i += gridDim.x * kRouteThreads)
    a.zero[i] = 0u;
  const int split = blockIdx.x % a.splits;
  const int eg = blockIdx.x / a.splits % a.egroups;
  const int tb = blockIdx.x / a.splits / a.egroups;
  const int t0 = tb * kRouteT, nt = min(kRouteT, a.T - t0);
  const int e = eg * 32 + lane;
  const int h_end = min(a.H, (split + 1) * a.rows_per_split);
  float acc[kRouteT] = {};
  for (int h0 = split * a.rows_per_split; h0 < h_end; h0 += kRouteChunk) {
    const int len = min(kRouteChunk, h_end - h0);
    __syncthreads();
    for (int i = threadIdx.x; i < kRouteT * len; i += kRouteThreads) {
      const int t = i / len, h = i - t * len;
      xs[t][h] = t < nt ? moe_h2f(a.X[static_cast<long long>(t0 + t) * a.ldx + h0 + h]) : 0.0f;
    }
    __syncthreads();
    if (e < a.E) {
      const uint16_t* w = a.Wr + static_cast<long long>(h0) * a.E + e;
#pragma unroll 8
      for (int h = warp; h < len; h += kRouteWarps) {
        const float wv = moe_h2f(__ldg(w + static_cast<long long>(h) * a.E));
#pragma unroll
        for (int t = 0; t < kRouteT; ++t) acc[t] = fmaf(xs[t][h], wv, acc[t]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < kRouteT; ++t) part[warp][t][lane] = acc[t];
  __syncthreads();
  if (threadIdx.x < 32 * kRouteT) {
    const int t = threadIdx.x >> 5;
    float s = 0.0f;
    for (int w = 0; w < kRouteWarps; ++w) s += part[w][t][lane];
    if (t < nt && e < a.E)
      __stcg(a.part + (static_cast<long long>(split) * a.T + t0 + t) * a.E + e, s);
  }
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    const unsigned int total = static_cast<unsigned int>(a.egroups * a.splits);
    last = atomicAdd(a.counters + tb, 1u) == total - 1u;
    if (last) a.counters[tb] = 0u;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  if (warp < nt) {
    const int t = t0 + warp;
    float* const l = logits + warp * a.E;
    for (int j = lane; j < a.E; j += 32) {
      float v[kMaxSplits], s = 0.0f;
#pragma unroll
      for (int k = 0; k < kMaxSplits; ++k)
        v[k] = k < a.splits ? __ldcg(a.part + (static_cast<long long>(k) * a.T + t) * a.E + j) : 0.0f;
#pragma unroll
      for (int k = 0; k < kMaxSplits; ++k) s += v[k];
      l[j] = s;
    }
    __syncwarp();
    int* const id = a.ids + static_cast<long long>(t) * a.topk;
    float* const p = a.probs + static_cast<long long>(t) * a.topk;
    select_experts(l, a.E, a.topk, a.renormalize, id, p);
    for (int k = lane; k < a.topk; k += 32) {
      if (a.ids_out) a.ids_out[static_cast<long long>(t) * a.topk + k] = id[k];
      if (a.probs_out) a.probs_out[static_cast<long long>(t) * a.topk + k] = p[k];
    }
  }
}

// ----------------------------------------------------------------- streaming
constexpr int kWeightBytes = 4 * 64 * 128;   // one k-block of a unit: 32 KB
constexpr int kMaxStages = 8;
constexpr int kLoaders = 4;                  // warps that stage token rows
constexpr int kEpi = 4;                      // epilogue warps of one accumulator buffer
constexpr int kStreamWarps = 2 + kLoaders + 2 * kEpi;
constexpr int kStreamThreads = 32 * kStreamWarps;
constexpr int kAccCols = 128;                // TMEM columns of one accumulator
constexpr int kTmemCols = 512;               // two buffers of two accumulators
constexpr int kSmemMax = 232448;
constexpr int kQueue = 4;                    // chunk numbers on their way to the consumers
constexpr int kBarBytes = 8 * (3 * kMaxStages + 5 + 2 * kQueue);
constexpr int kTopPad = 8;                   // words to a row's magnitude: in one sector the
                                             // maxima of eight rows took 0.6 us longer
constexpr int kScales = 8;                   // chunks whose rows' scales are kept
static_assert(kScales > kQueue, "the chunk an epilogue warp is at, and a queue of later ones");
constexpr int kFixedBytes = (kBarBytes + 4 * kQueue + 8 + 4 * kScales * kBlockT + 15) / 16 * 16;

struct StreamArgs {
  const uint16_t* X;
  long long ldx;
  uint16_t* Y;
  long long ldy;
  const int* ids;          // [T][topk]
  const float* probs;
  int T, H, I, E, topk;
  float beta;
  int up_tiles, up_kb, down_tiles, down_kb;
  int stages, stage_bytes;
  float* hid;              // [T * topk][I]
  unsigned int* top;       // [T * topk][kTopPad]: the rows' largest finite magnitude, as bits
  float* up_part;          // by unit and chunk: [acc][token][128]
  float* z;                // [T * topk][chunk][H]
  unsigned int* queue;     // chunks taken so far
  unsigned int* done;      // down chunks finished, by epilogue warp
  unsigned int* ready;     // [active expert] up units finished, by epilogue warp
  unsigned int* counters;  // [up unit][epilogue warp] chunks arrived
  unsigned long long wait_limit_ns;
  DeviceStatus* status;
};

// Chunks per unit of `kb` k-blocks, for `active` experts of `tiles` units each
// and `pairs` (token, expert) pairs.  A chunk has at least
//   * 1/8 of an SM's even share, so that the last ones to finish are short
//     without the partial sums growing for nothing,
//   * 4 k-blocks (128 KB, ~2.8 us of an SM's share of HBM): publishing a chunk's
//     sums and counting it in takes the two groups of epilogue warps about 2 us
//     each (with 2 k-blocks they fell behind the stream by 10 us),
//   * and one more for each token an expert has, for the 1 KB of sums per token
//     written and read back (a quarter of a k-block per token instead: 64 tokens
//     at 8 experts of 4096 x 1408, top 2, 110 us against 72), but for at most a
//     third of the unit, so that a few busy experts still reach every SM (60
//     tokens at 6 experts of 3008 x 1600, top 4, 103 us without, 82 with it).
__host__ __device__ inline int chunks_of(int active, int tiles, int kb, int pairs, int ctas) {
  const int share = active * tiles * kb / (8 * ctas);
  const int tokens = pairs / active, least = 4 + (tokens < kb / 3 ? tokens : kb / 3);
  const int len = share > least ? share : least;
  return len >= kb ? 1 : (kb + len - 1) / len;
}

// The chunks of a launch: [0, up) then [up, up + down).
struct Work {
  int up_tiles, up_kb, up_chunks, down_tiles, down_kb, down_chunks;
  int up, total;
};

struct Chunk {
  int down, unit, q, tile, c, kb0, kb1;
};

__device__ __forceinline__ Chunk chunk_at(const Work& w, int id) {
  Chunk t;
  t.down = id >= w.up;
  if (t.down) id -= w.up;
  const int n = t.down ? w.down_chunks : w.up_chunks, kb = t.down ? w.down_kb : w.up_kb;
  const int tiles = t.down ? w.down_tiles : w.up_tiles;
  t.unit = id / n;
  t.c = id - t.unit * n;
  t.kb0 = t.c * kb / n;
  t.kb1 = (t.c + 1) * kb / n;
  t.q = t.unit / tiles;
  t.tile = t.unit - t.q * tiles;
  return t;
}

__host__ __device__ inline int round_up(int x, int m) { return (x + m - 1) / m * m; }

// Counts in at GPU scope after __syncwarp(): what the warp's lanes wrote before
// is released with it (and acquired by whoever reads the count).
__device__ __forceinline__ unsigned int add_acq_rel(unsigned int* p) {
  unsigned int before;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(before) : "l"(p) : "memory");
  return before;
}

__device__ __forceinline__ void add_release(unsigned int* p) {
  asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(p) : "memory");
}

__global__ void __launch_bounds__(kStreamThreads, 1)
    moe_stream_kernel(const __grid_constant__ CUtensorMap tm1,
                      const __grid_constant__ CUtensorMap tm2, const StreamArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const base_ptr = smem_raw + (base - raw);
  const int S = a.stages;
  const int warp = warp_id_uniform(), lane = static_cast<int>(lane_id());
  const int cta = blockIdx.x, ctas = gridDim.x;
  const int P = a.T * a.topk;

  // after the ring: barriers, the chunk queue, then the routing lists
  uint8_t* const tail = base_ptr + static_cast<size_t>(S) * a.stage_bytes;
  const uint32_t bars = base + static_cast<uint32_t>(S * a.stage_bytes);
  auto full_bar = [&](int s) { return bars + 8u * s; };                     // weights landed
  auto tok_bar = [&](int s) { return bars + 8u * (kMaxStages + s); };       // token rows staged
  auto empty_bar = [&](int s) { return bars + 8u * (2 * kMaxStages + s); };
  auto accf_bar = [&](uint32_t b) { return bars + 8u * (3 * kMaxStages + b); };
  auto acce_bar = [&](uint32_t b) { return bars + 8u * (3 * kMaxStages + 2 + b); };
  const uint32_t done_bar = bars + 8u * (3 * kMaxStages + 4);
  auto qfull_bar = [&](int i) { return bars + 8u * (3 * kMaxStages + 5 + i); };
  auto qempty_bar = [&](int i) { return bars + 8u * (3 * kMaxStages + 5 + kQueue + i); };
  volatile int* const s_queue = reinterpret_cast<int*>(tail + kBarBytes);
  uint32_t* const misc = reinterpret_cast<uint32_t*>(tail + kBarBytes + 4 * kQueue);
  // by chunk: what takes the scale of a row of hid back
  volatile float* const s_down = reinterpret_cast<float*>(misc + 2);   // [kScales][kBlockT]
  uint16_t* const s_ids = reinterpret_cast<uint16_t*>(tail + kFixedBytes);   // expert of a pair
  const int P8 = round_up(P, 8), E2 = round_up(a.E, 2);
  uint16_t* const s_list = s_ids + P8;    // pairs by (expert, pair)
  uint16_t* const s_pos = s_list + P8;    // place of a pair in s_list
  uint16_t* const s_off = s_pos + P8;     // first place of expert e
  uint16_t* const s_act = s_off + E2;     // active experts in order
  int* const s_cnt = reinterpret_cast<int*>(s_act + E2);   // tokens of expert e

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1u);
      mbar_init(tok_bar(s), 1u);
      mbar_init(empty_bar(s), 1u);
    }
    for (uint32_t b = 0; b < 2; ++b) {
      mbar_init(accf_bar(b), 2u);   // the products, and the MMA thread for the scales
      mbar_init(acce_bar(b), static_cast<uint32_t>(kEpi));
    }
    mbar_init(done_bar, 1u);
    for (int i = 0; i < kQueue; ++i) {
      mbar_init(qfull_bar(i), 1u);
      mbar_init(qempty_bar(i), static_cast<uint32_t>(1 + kLoaders + 2 * kEpi));
    }
    fence_barrier_init();
    fence_proxy_async_smem();
    prefetch_tensormap(&tm1);
    prefetch_tensormap(&tm2);
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(misc), kTmemCols);
    tmem_relinquish();
  }
  for (int e = threadIdx.x; e < a.E; e += kStreamThreads) s_cnt[e] = 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(misc);
  griddep_wait();   // the routing kernel's ids, p and zeroed counters
  int next_id = 0;  // warp 0, lane 0: the chunk taken last
  if (threadIdx.x == 0) next_id = static_cast<int>(atomicAdd(a.queue, 1u));

  // ---- lists: every expert's pairs in order
  for (int i = threadIdx.x; i < P8; i += kStreamThreads) {
    int e = 0xFFFF;
    if (i < P) {
      e = __ldcg(a.ids + i);
      atomicAdd(s_cnt + e, 1);
    }
    s_ids[i] = static_cast<uint16_t>(e);
  }
  __syncthreads();
  if (warp == 0) {
    int off = 0, act = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + lane;
      const int n = e < a.E ? s_cnt[e] : 0;
      int incl = n;
      for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += v;
      }
      const unsigned int some = __ballot_sync(0xffffffffu, n > 0);
      if (e < a.E) {
        s_off[e] = static_cast<uint16_t>(off + incl - n);
        if (n > 0)
          s_act[act + __popc(some & ((1u << lane) - 1u))] = static_cast<uint16_t>(e);
      }
      off += __shfl_sync(0xffffffffu, incl, 31);
      act += __popc(some);
    }
    if (lane == 0) misc[1] = static_cast<uint32_t>(act);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < P; i += kStreamThreads) {
    // place: the expert's first one plus its pairs before this one
    const uint32_t e = s_ids[i], key = e * 0x10001u;
    uint32_t bits = 0;
    int j = 0;
    for (; j + 8 <= i; j += 8) {
      const uint4 w = *reinterpret_cast<const uint4*>(s_ids + j);
      bits += __popc(__vcmpeq2(w.x, key)) + __popc(__vcmpeq2(w.y, key)) +
              __popc(__vcmpeq2(w.z, key)) + __popc(__vcmpeq2(w.w, key));
    }
    int pos = s_off[e] + static_cast<int>(bits >> 4);
    for (; j < i; ++j) pos += s_ids[j] == e;
    s_pos[i] = static_cast<uint16_t>(pos);
    s_list[pos] = static_cast<uint16_t>(i);
  }
  __syncthreads();
  const int active = static_cast<int>(misc[1]);
  Work w;
  w.up_tiles = a.up_tiles;
  w.up_kb = a.up_kb;
  w.up_chunks = chunks_of(active, a.up_tiles, a.up_kb, P, ctas);
  w.down_tiles = a.down_tiles;
  w.down_kb = a.down_kb;
  w.down_chunks = chunks_of(active, a.down_tiles, a.down_kb, P, ctas);
  w.up = active * w.up_tiles * w.up_chunks;
  w.total = w.up + active * w.down_tiles * w.down_chunks;
  const unsigned long long limit = a.wait_limit_ns;
  DeviceStatus* const st = a.status;

  // A consumer's next chunk number, -1 at the end (or when a wait gave up).
  int qi = 0;
  uint32_t qphase = 0;
  auto next_chunk = [&]() -> int {   // one thread
    if (!wait_parity(qfull_bar(qi), qphase, limit, st, 50)) return -1;
    const int id = s_queue[qi];
    mbar_arrive(qempty_bar(qi));
    if (++qi == kQueue) {
      qi = 0;
      qphase ^= 1u;
    }
    return id;
  };
  auto next_chunk_warp = [&]() -> int {   // whole warp
    int id = 0;
    if (lane == 0) id = next_chunk();
    return __shfl_sync(0xffffffffu, id, 0);
  };

  if (warp == 0) {
    // ------------------------------------------- chunk numbers, weights (TMA)
    if (lane == 0) {
      const uint64_t policy = l2_evict_first_policy();
      int stage = 0;
      uint32_t phase = 0, issued = 0;
      bool ok = true;
      for (;;) {
        const int id = ok && next_id < w.total ? next_id : -1;
        if (!wait_parity(qempty_bar(qi), qphase ^ 1u, limit, st, 39)) break;
        s_queue[qi] = id;
        mbar_arrive(qfull_bar(qi));
        if (++qi == kQueue) {
          qi = 0;
          qphase ^= 1u;
        }
        if (id < 0) break;
        next_id = static_cast<int>(atomicAdd(a.queue, 1u));   // back by the end of this chunk
        const Chunk t = chunk_at(w, id);
        const int e = s_act[t.q];
        // columns of the four boxes; one that lies past the matrix is skipped
        int col[4], n = 0;
        bool use[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          if (t.down) {
            col[b] = t.tile * 256 + b * 64;
            use[b] = col[b] < a.H;
          } else {
            const int j = t.tile * 128 + (b & 1) * 64;
            use[b] = j < a.I;
            col[b] = (b >> 1) * a.I + j;
          }
          n += use[b];
        }
        const CUtensorMap* const tm = t.down ? &tm2 : &tm1;
        for (int kb = t.kb0; kb < t.kb1; ++kb) {
          if (!wait_parity(empty_bar(stage), phase ^ 1u, limit, st, 40)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(full_bar(stage), static_cast<uint32_t>(n * 8192));
          const uint32_t dst = base + static_cast<uint32_t>(stage * a.stage_bytes);
#pragma unroll
          for (int b = 0; b < 4; ++b)
            if (use[b])
              tma_load_3d_hint(dst + b * 8192, tm, full_bar(stage), col[b], kb * 64, e, policy);
          ++issued;
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // loads still in flight must land before the CTA exits
      const uint32_t n = min(issued, static_cast<uint32_t>(S));
      for (uint32_t i = issued - n; i < issued; ++i)
        settle_wait(full_bar(static_cast<int>(i % S)), (i / S) & 1u, st, 41);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, local = 0;
      bool ok = true;
      for (int id; ok && (id = next_chunk()) >= 0;) {
        const Chunk t = chunk_at(w, id);
        const int n = s_cnt[s_act[t.q]];
        const int cols = t.down ? 2 * round_up(n, 8) : round_up(n, 16);
        const uint32_t idesc = make_idesc(0u, 128u, static_cast<uint32_t>(cols), 1u, 0u);
        const uint32_t buf = local & 1u;
        if (!wait_parity(acce_bar(buf), ((local >> 1) & 1u) ^ 1u, limit, st, 42)) break;
        tc_fence_after();
        const uint32_t d0 = tmem + buf * (2 * kAccCols);
        for (int kb = t.kb0; kb < t.kb1; ++kb) {
          if (!wait_parity(full_bar(stage), phase, limit, st, 43) ||
              !wait_parity(tok_bar(stage), phase, limit, st, 44)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t w0 = base + static_cast<uint32_t>(stage * a.stage_bytes);
          const uint32_t x0 = w0 + kWeightBytes;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t bd = smem_desc_sw128(x0 + kk * 32, 16u, 1024u);
            const uint32_t acc = (kb > t.kb0 || kk > 0) ? 1u : 0u;
            mma_f16_ss(d0, smem_desc_sw128(w0 + kk * 2048, 8192u, 1024u), bd, idesc, acc);
            mma_f16_ss(d0 + kAccCols, smem_desc_sw128(w0 + 16384 + kk * 2048, 8192u, 1024u), bd,
                       idesc, acc);
          }
          mma_commit(empty_bar(stage));
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        mma_commit(accf_bar(buf));
        mbar_arrive(accf_bar(buf));
        ++local;
      }
      mma_commit(done_bar);
      settle_wait(done_bar, 0u, st, 45);
    }
    __syncwarp();
  } else if (warp < 2 + kLoaders) {
    // ---------------------------------------------------------- token rows
    // Loader l stages the k-blocks l, l + 4, ... of the CTA's sequence: rows
    // of X for up; for down the hi parts of the rows of hid, then (from the next
    // multiple of 8) the lo parts.  Rows past them are left as they are: their
    // columns of the product are never read.
    const int l = warp - 2;
    int stage = 0, seq = 0, place = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int id; ok && (id = next_chunk_warp()) >= 0; ++place) {
      const Chunk t = chunk_at(w, id);
      const int e = s_act[t.q];
      const int n = s_cnt[e], off = s_off[e], n8 = round_up(n, 8);
      unsigned int top[2] = {};   // of rows lane and lane + 32 (kBlockT in all)
      if (t.down) {   // hid of the expert's pairs is written
        if (lane == 0)
          ok = wait_count(a.ready + t.q, static_cast<unsigned int>(kEpi * w.up_tiles), limit, st, 46);
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        __syncwarp();
        if (!ok) break;
#pragma unroll
        for (int u = 0; u < 2; ++u)
          if (lane + 32 * u < n) top[u] = __ldcg(a.top + (off + lane + 32 * u) * kTopPad);
      }
      for (int kb = t.kb0; kb < t.kb1; ++kb, ++seq) {
        if ((seq & (kLoaders - 1)) == l) {
          if (!wait_parity(empty_bar(stage), phase ^ 1u, limit, st, 47)) {
            ok = false;
            break;
          }
          uint8_t* const dst = base_ptr + static_cast<size_t>(stage) * a.stage_bytes + kWeightBytes;
          if (t.down) {
            // four entries at a time
            for (int i0 = 0; i0 < n * 16; i0 += 32 * 4) {
              float4 v[4];
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const int i = i0 + 32 * u + lane;
                const int r = i >> 4, k = kb * 64 + (i & 15) * 4;
                v[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (r < n && k < a.I)
                  v[u] = __ldcg(reinterpret_cast<const float4*>(
                      a.hid + static_cast<long long>(off + r) * a.I + k));
              }
              // (not before the loads: the compiler would wait for top first)
              asm volatile("" : "+r"(top[0]), "+r"(top[1]));
              const float mine = moe_scale(i0 < 512 ? top[0] : top[1]);
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const int i = i0 + 32 * u + lane;
                const int r = i >> 4, c = i & 15;
                // (rows i0 / 16 .. i0 / 16 + 7 are on one side of 32)
                const float up = __shfl_sync(0xffffffffu, mine, r & 31);
                if (r < n) {
                  uint2 hi, lo;
                  moe_split4(v[u], up, hi, lo);
                  // n8 is a multiple of 8
                  uint8_t* const o = dst + r * 128 + (((c >> 1) ^ (r & 7)) << 4) + 8 * (c & 1);
                  *reinterpret_cast<uint2*>(o) = hi;
                  *reinterpret_cast<uint2*>(o + n8 * 128) = lo;
                }
              }
            }
            if (kb == t.kb0)
#pragma unroll
              for (int u = 0; u < 2; ++u)
                s_down[place % kScales * kBlockT + lane + 32 * u] =
                    moe_unscale(moe_scale(top[u]));
          } else {
            for (int i0 = 0; i0 < n * 8; i0 += 32 * 4) {
              uint4 v[4];
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const int i = i0 + 32 * u + lane;
                const int r = i >> 3, k = kb * 64 + (i & 7) * 8;
                v[u] = make_uint4(0u, 0u, 0u, 0u);
                if (r < n && k < a.H)
                  v[u] = __ldg(reinterpret_cast<const uint4*>(
                      a.X + static_cast<long long>(s_list[off + r] / a.topk) * a.ldx + k));
              }
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const int i = i0 + 32 * u + lane;
                const int r = i >> 3, c = i & 7;
                if (r < n) *reinterpret_cast<uint4*>(dst + r * 128 + ((c ^ (r & 7)) << 4)) = v[u];
              }
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(tok_bar(stage));
        }
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else {
    // ---------------------------------------------------------- epilogue
    const int quad = warp & 3;                 // TMEM lanes 32 quad ..
    const int col = 32 * quad + lane;          // this thread's column of a 128-wide accumulator
    const uint32_t buf = static_cast<uint32_t>(warp - 2 - kLoaders) / kEpi;   // every other chunk
    uint32_t local = 0;
    for (int id; (id = next_chunk_warp()) >= 0; ++local) {
      if ((local & 1u) != buf) continue;
      const Chunk t = chunk_at(w, id);
      const int e = s_act[t.q];
      const int n = s_cnt[e], off = s_off[e], n8 = round_up(n, 8);
      if (!wait_parity(accf_bar(buf), (local >> 1) & 1u, limit, st, 48)) break;
      tc_fence_after();
      const uint32_t d0 = tmem + (static_cast<uint32_t>(32 * quad) << 16) + buf * (2 * kAccCols);
      // hid of 8 tokens at column j, and the largest of the warp's columns
      const int j = t.tile * 128 + col;
      auto store_hid = [&](int r0, const float (&g)[8], const float (&u)[8]) {
        unsigned int top = 0u;   // lane i: of token r0 + i
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          // for all lanes or none: one jump past the code of tokens that are not
          // there (a jump for each fetched 0.7 us of code at one token)
          if (r0 + i >= n) break;
          float h = 0.0f;
          if (j < a.I) {
            h = g[i] / (1.0f + expf(-g[i])) * u[i];
            a.hid[static_cast<long long>(off + r0 + i) * a.I + j] = h;
          }
          const unsigned int most = __reduce_max_sync(0xffffffffu, moe_finite_bits(h));
          if (lane == i) top = most;
        }
        if (lane < 8 && top != 0u) atomicMax(a.top + (off + r0 + lane) * kTopPad, top);
      };
      float* const unit_part =
          t.down ? nullptr
                 : a.up_part + (static_cast<long long>(off) * w.up_tiles + t.tile * n) *
                                   w.up_chunks * 256 + col;
      for (int r0 = 0; r0 < n; r0 += 8) {
        float v0[8], v1[8];
        uint32_t g[8], h[8];
        tmem_ld_32x32b_x8(d0 + r0, g);
        tmem_ld_32x32b_x8(d0 + kAccCols + r0, h);
        tmem_wait_ld2(g, h);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v0[i] = __uint_as_float(g[i]);
          v1[i] = __uint_as_float(h[i]);
        }
        if (t.down) {
          // hi and lo parts
          tmem_ld_32x32b_x8(d0 + n8 + r0, g);
          tmem_ld_32x32b_x8(d0 + kAccCols + n8 + r0, h);
          tmem_wait_ld2(g, h);
          const int c0 = t.tile * 256 + col;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (r0 + i < n) {
              const float down = s_down[local % kScales * kBlockT + r0 + i];
              float* o = a.z + (static_cast<long long>(off + r0 + i) * w.down_chunks + t.c) * a.H;
              if (c0 < a.H) __stcg(o + c0, down * moe_join(v0[i], __uint_as_float(g[i])));
              if (c0 + 128 < a.H)
                __stcg(o + c0 + 128, down * moe_join(v1[i], __uint_as_float(h[i])));
            }
        } else if (w.up_chunks == 1) {
          store_hid(r0, v0, v1);
        } else {
          float* const mine = unit_part + t.c * n * 256;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (r0 + i < n) {
              __stcg(mine + (r0 + i) * 128, v0[i]);
              __stcg(mine + (n + r0 + i) * 128, v1[i]);
            }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acce_bar(buf));   // the accumulators may be overwritten
      if (t.down) {
        if (lane == 0) add_release(a.done);
        continue;
      }
      bool last = true;
      if (w.up_chunks > 1) {
        // the last of the unit's chunks to arrive adds them up in k order
        unsigned int before = 0;
        if (lane == 0) before = add_acq_rel(a.counters + t.unit * kEpi + quad);
        last = __shfl_sync(0xffffffffu, before, 0) == static_cast<unsigned int>(w.up_chunks - 1);
        __syncwarp();
        if (last) {
          for (int r0 = 0; r0 < n; r0 += 8) {
            float v0[8] = {}, v1[8] = {};
            if (n - r0 <= 2) {
              // few tokens: the loads of eight chunks in flight
              for (int c0 = 0; c0 < w.up_chunks; c0 += 8) {
                float x[8][4];
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                  const float* src = unit_part + static_cast<long long>(c0 + c) * n * 256;
#pragma unroll
                  for (int i = 0; i < 2; ++i) {
                    const bool in = c0 + c < w.up_chunks && r0 + i < n;
                    x[c][i] = in ? __ldcg(src + (r0 + i) * 128) : 0.0f;
                    x[c][2 + i] = in ? __ldcg(src + (n + r0 + i) * 128) : 0.0f;
                  }
                }
#pragma unroll
                for (int c = 0; c < 8; ++c)
#pragma unroll
                  for (int i = 0; i < 2; ++i) {
                    v0[i] += x[c][i];
                    v1[i] += x[c][2 + i];
                  }
              }
            } else {
#pragma unroll 4
              for (int c = 0; c < w.up_chunks; ++c) {
                const float* src = unit_part + static_cast<long long>(c) * n * 256;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  if (r0 + i < n) {
                    v0[i] += __ldcg(src + (r0 + i) * 128);
                    v1[i] += __ldcg(src + (n + r0 + i) * 128);
                  }
              }
            }
            store_hid(r0, v0, v1);
          }
          __syncwarp();
        }
      }
      if (last && lane == 0) add_release(a.ready + t.q);
    }
  }

  // ---- sum: z of every pair is written.  `group` warps share a (token, 32
  // columns) item, each with its own k; their terms meet in shared memory.
  __syncthreads();   // the roles are done: the ring's memory is free, TMEM is read
  bool* const s_ok = reinterpret_cast<bool*>(misc + 1);
  if (threadIdx.x == 0)
    *s_ok = wait_count(a.done, static_cast<unsigned int>(kEpi * (w.total - w.up)), limit, st, 49);
  __syncthreads();
  if (*s_ok) {
    const int strips = (a.H + 31) / 32, items = a.T * strips;
    int group = 1;   // 8 warps of the CTA take part
    while (group < 8 && 2 * group * items <= 8 * ctas) group *= 2;
    const int per = 8 / group;
    float* const s_sum = reinterpret_cast<float*>(base_ptr);   // [8][32]
    const int g = warp % group;
    for (int it0 = cta * per; it0 < items; it0 += ctas * per) {
      const int it = it0 + warp / group;
      const int t = it / strips, c = (it - t * strips) * 32 + lane;
      const bool mine = warp < 8 && it < items && c < a.H;
      float y = 0.0f;
      if (mine) {
        for (int k0 = g; k0 < a.topk; k0 += 4 * group) {
          float z[4], p[4];
          const float* src[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int k = k0 + u * group;
            const int pair = t * a.topk + min(k, a.topk - 1);
            src[u] = a.z + static_cast<long long>(s_pos[pair]) * w.down_chunks * a.H + c;
            p[u] = k < a.topk ? __ldcg(a.probs + pair) : 0.0f;
            z[u] = k < a.topk ? __ldcg(src[u]) : 0.0f;
          }
          for (int ch = 1; ch < w.down_chunks; ++ch)
#pragma unroll
            for (int u = 0; u < 4; ++u)
              if (k0 + u * group < a.topk) z[u] += __ldcg(src[u] + static_cast<long long>(ch) * a.H);
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (k0 + u * group < a.topk) y = fmaf(p[u], z[u], y);
        }
      }
      if (group > 1) {
        if (warp < 8) s_sum[warp * 32 + lane] = y;
        __syncthreads();
        if (g == 0 && mine)
          for (int u = 1; u < group; ++u) y += s_sum[(warp + u) * 32 + lane];
        __syncthreads();
      }
      if (g == 0 && mine) {
        uint16_t* o = a.Y + static_cast<long long>(t) * a.ldy + c;
        *o = moe_f2h(a.beta != 0.0f ? fmaf(a.beta, moe_h2f(*o), y) : y);
      }
    }
  }
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

bool moe_stream_fits(const MoeArgs& m) {
  const uintptr_t ptrs = reinterpret_cast<uintptr_t>(m.X) | reinterpret_cast<uintptr_t>(m.W1) |
                         reinterpret_cast<uintptr_t>(m.W2);
  // the rows of X, W1 (2I halves) and W2 (H) on the 16-byte grid
  if ((ptrs & 15u) != 0 || m.H % 8 != 0 || m.I % 8 != 0 || m.ldx % 8 != 0 || m.I == 0) return false;
  // k-blocks are counted in 32 bits
  const long long kb = (m.H / 64 + 1ll) * (m.I / 64 + 1ll);
  return kb * m.E < (1ll << 28);
}

int moe_stream(const MoeArgs& m, int sms, DeviceStatus* st, unsigned long long limit_ns,
               cudaStream_t stream) {
  CUtensorMap tm1{}, tm2{};
  if (int rc = encode_map_f16_stack(&tm1, m.W1, m.H, 2 * m.I, 2ll * m.I, m.E, 2ll * m.I * m.H, 64, 64))
    return rc;
  if (int rc = encode_map_f16_stack(&tm2, m.W2, m.I, m.H, m.H, m.E, 1ll * m.H * m.I, 64, 64))
    return rc;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return GEMM_ERR_CUDA;
  static bool configured[64] = {};
  if (dev < 64 && !configured[dev]) {
    if (cudaFuncSetAttribute(moe_stream_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSmemMax) != cudaSuccess)
      return GEMM_ERR_CUDA;
    configured[dev] = true;
  }
  for (int t0 = 0; t0 < m.T; t0 += kBlockT) {
    const int T = std::min(kBlockT, m.T - t0);
    const int P = T * m.topk;
    StreamArgs s{};
    s.T = T;
    s.H = m.H;
    s.I = m.I;
    s.E = m.E;
    s.topk = m.topk;
    s.beta = m.beta;
    s.X = m.X + static_cast<long long>(t0) * m.ldx;
    s.ldx = m.ldx;
    s.Y = m.Y + static_cast<long long>(t0) * m.ldy;
    s.ldy = m.ldy;
    s.up_tiles = (m.I + 127) / 128;
    s.up_kb = (m.H + 63) / 64;
    s.down_tiles = (m.H + 255) / 256;
    s.down_kb = (m.I + 63) / 64;
    s.wait_limit_ns = limit_ns;
    s.status = st;
    // token rows of a stage: X rows padded to 16, or hi and lo rows padded to 8
    const int rows = std::max((T + 15) / 16 * 16, 2 * ((T + 7) / 8 * 8));
    s.stage_bytes = kWeightBytes + rows * 128;
    const int lists = kFixedBytes + 2 * (3 * round_up(P, 8) + 2 * round_up(m.E, 2)) + 4 * m.E;
    s.stages = std::min(kMaxStages, (kSmemMax - 1024 - lists) / s.stage_bytes);
    if (s.stages < 2) return GEMM_ERR_ARG;

    RouteArgs r{};
    r.X = s.X;
    r.Wr = m.Wr;
    r.ldx = m.ldx;
    r.T = T;
    r.H = m.H;
    r.E = m.E;
    r.topk = m.topk;
    r.renormalize = m.renormalize;
    r.egroups = (m.E + 31) / 32;
    r.tblocks = (T + kRouteT - 1) / kRouteT;
    // K slices: about one CTA per SM in all, at most 16, none under 32 rows
    const int want = std::max(1, std::min({sms / (r.egroups * r.tblocks), kMaxSplits, m.H / 32}));
    r.rows_per_split = (m.H + want - 1) / want;
    r.splits = (m.H + r.rows_per_split - 1) / r.rows_per_split;

    // most chunks of a unit over the numbers of experts that may be active
    const int experts = std::min(m.E, P);
    int up_chunks = 1, down_chunks = 1;
    for (int n = 1; n <= experts; ++n) {
      up_chunks = std::max(up_chunks, chunks_of(n, s.up_tiles, s.up_kb, P, sms));
      down_chunks = std::max(down_chunks, chunks_of(n, s.down_tiles, s.down_kb, P, sms));
    }
    const long long units = 1ll * experts * s.up_tiles;
    const size_t b_part = round256(4 * static_cast<size_t>(r.splits) * T * m.E);
    const size_t b_ids = round256(4 * static_cast<size_t>(P));
    const size_t b_hid = round256(4 * static_cast<size_t>(P) * m.I);
    const size_t b_z = round256(4 * static_cast<size_t>(P) * down_chunks * m.H);
    const size_t b_ws = round256(4 * static_cast<size_t>(P) * s.up_tiles * up_chunks * 256);
    const size_t n_zero = static_cast<size_t>(units) * kEpi + experts + kTopPad * (P + 1);
    const size_t b_cnt = round256(4 * n_zero);
    void *buf = nullptr, *zero = nullptr;
    if (int rc = routed_scratch(stream, b_part + 2 * b_ids + b_hid + b_z + b_ws + b_cnt, &buf,
                                4 * static_cast<size_t>(kBlockT / kRouteT), &zero))
      return rc;
    uint8_t* b = static_cast<uint8_t*>(buf);
    auto take = [&](size_t n) {
      uint8_t* p = b;
      b += n;
      return p;
    };
    r.part = reinterpret_cast<float*>(take(b_part));
    r.ids = reinterpret_cast<int*>(take(b_ids));
    r.probs = reinterpret_cast<float*>(take(b_ids));
    s.hid = reinterpret_cast<float*>(take(b_hid));
    s.z = reinterpret_cast<float*>(take(b_z));
    s.up_part = reinterpret_cast<float*>(take(b_ws));
    s.queue = reinterpret_cast<unsigned int*>(take(b_cnt));
    s.done = s.queue + 1;
    s.top = s.queue + kTopPad;
    s.ready = s.top + kTopPad * P;
    s.counters = s.ready + experts;
    s.ids = r.ids;
    s.probs = r.probs;
    r.counters = static_cast<unsigned int*>(zero);
    r.zero = s.queue;
    r.nzero = static_cast<int>(n_zero);
    r.ids_out = m.ids ? m.ids + static_cast<long long>(t0) * m.topk : nullptr;
    r.probs_out = m.probs ? m.probs + static_cast<long long>(t0) * m.topk : nullptr;

    const size_t route_smem = 4 * static_cast<size_t>(kRouteT) * m.E;
    moe_logits_kernel<<<r.tblocks * r.egroups * r.splits, kRouteThreads, route_smem, stream>>>(r);
    if (counted_launch(cudaGetLastError()) != cudaSuccess) return GEMM_ERR_CUDA;

    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(sms), 1, 1);
    cfg.blockDim = dim3(kStreamThreads, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(s.stages) * s.stage_bytes + lists + 1024;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, moe_stream_kernel, tm1, tm2, s) != cudaSuccess)
      return GEMM_ERR_CUDA;
    note_launch();
  }
  set_last_path("moe.stream");
  return GEMM_OK;
}

}  // namespace gb300
