// moe_stream.cu -- the mixture-of-experts layer for a few tokens in two
// kernels that read each chosen expert's weights once.
//
//   moe_logits_kernel  l = x Wr as K slices over many CTAs; the CTA that ends a
//                      block of four tokens adds the slices up in order, picks
//                      the topk experts and writes ids and p.
//   moe_stream_kernel  one CTA per SM, all resident (cooperative launch):
//     up    hid = silu(x W1g) .* (x W1u) of every (token, expert) pair
//     down  z = hid W2 per pair
//     sum   y = sum_k p_k z_k + beta y
//
// With n tokens at an expert a weight takes part in n multiply-adds, far fewer
// than the ~280 per byte at which the tensor cores bind: the time is that of
// streaming the weights from HBM.  So the weights are the M operand: a unit is
// 128 + 128 columns of an expert's matrix (gate and up columns j, or 256
// columns of W2) in two TMEM accumulators, the expert's tokens the N operand
// (N = 16..128), and a k-block is 64 rows of the matrix, 32 KB by TMA.  All
// k-blocks of all units are shared out evenly: CTA c takes [c, c+1) * total /
// CTAs, cut at unit boundaries into pieces.  A piece that is not a whole unit
// publishes fp32 partial sums; the last piece of an up unit to arrive adds them
// in k order (so the result does not depend on which that is), the sum step
// does so for down units.  The weights do not depend on the grid-wide barrier
// between up and down, so W2 streams into the ring across it; only the warps
// that stage hid wait.
//
// hid is kept as two halves, hi + lo (22 significant bits), staged as separate
// rows of the N operand and added up after the products, so the layer's only
// rounding to half is that of Y.  A token's columns never mix with another's,
// and a pair's partial results are read only for its own token.
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
constexpr int kMaxPairs = kBlockT * kMoeMaxTopk;

// ------------------------------------------------------------------ routing
constexpr int kRouteThreads = 256;
constexpr int kRouteWarps = kRouteThreads / 32;
constexpr int kRouteT = 4;                   // tokens per CTA
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
  extern __shared__ float logits[];          // [kRouteT][E], then the marks
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
    uint8_t* const taken = reinterpret_cast<uint8_t*>(logits + kRouteT * a.E) + warp * a.E;
    for (int j = lane; j < a.E; j += 32) {
      float s = 0.0f;
      for (int k = 0; k < a.splits; ++k)
        s += __ldcg(a.part + (static_cast<long long>(k) * a.T + t) * a.E + j);
      l[j] = s;
    }
    __syncwarp();
    int* const id = a.ids + static_cast<long long>(t) * a.topk;
    float* const p = a.probs + static_cast<long long>(t) * a.topk;
    select_experts(l, taken, a.E, a.topk, a.renormalize, id, p);
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
constexpr int kEpi = 4;                      // epilogue warps
constexpr int kStreamWarps = 2 + kLoaders + kEpi;
constexpr int kStreamThreads = 32 * kStreamWarps;
constexpr int kAccCols = 128;                // TMEM columns of one accumulator
constexpr int kTmemCols = 512;               // two buffers of two accumulators
constexpr int kSmemMax = 232448;

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
  uint16_t* hid;           // [2][T * topk][I]: hi, lo
  float* z;                // [T * topk][H], whole down units
  float* part;             // [phase][CTA][first / last piece][acc][token][128]
  int part_tokens;
  unsigned int* counters;  // [up unit][4 epilogue warps]
  unsigned int* bars;      // arrivals after up, after down
  unsigned long long wait_limit_ns;
  DeviceStatus* status;
};

// A CTA's share of a phase: k-blocks [beg, end) of the phase's tot = active
// experts * tiles * kb.  The first `workers` CTAs have one, at least kMinKb
// k-blocks long (none is empty, so the owners of a unit are consecutive CTAs).
constexpr int kMinKb = 2;
struct Phase {
  long long tot, beg, end;
  int tiles, kb, workers;
};

struct Piece {
  int q, tile, kb0, kb1;
  long long unit;
};

__device__ __forceinline__ Phase phase_of(long long active, int tiles, int kb, int cta, int ctas) {
  Phase p;
  p.tiles = tiles;
  p.kb = kb;
  p.tot = active * tiles * kb;
  p.workers = static_cast<int>(min(static_cast<long long>(ctas), max(1ll, p.tot / kMinKb)));
  p.beg = cta < p.workers ? cta * p.tot / p.workers : 0;
  p.end = cta < p.workers ? (cta + 1) * p.tot / p.workers : 0;
  return p;
}

__device__ __forceinline__ Piece piece_at(const Phase& p, long long x) {
  Piece t;
  t.unit = x / p.kb;
  t.kb0 = static_cast<int>(x - t.unit * p.kb);
  t.kb1 = static_cast<int>(min(static_cast<long long>(p.kb), t.kb0 + (p.end - x)));
  t.q = static_cast<int>(t.unit / p.tiles);
  t.tile = static_cast<int>(t.unit - static_cast<long long>(t.q) * p.tiles);
  return t;
}

// The CTA whose share holds k-block x.
__device__ __forceinline__ int owner_of(const Phase& p, long long x) {
  return static_cast<int>(((x + 1) * p.workers - 1) / p.tot);
}

// Partial sums of CTA w for a unit that starts at k-block u0: its first piece
// (slot 0) when its share starts inside the unit, else its last one (slot 1).
__device__ __forceinline__ float* part_of(const StreamArgs& a, const Phase& p, int phase, int w,
                                          int ctas, long long u0) {
  const int slot = w * p.tot / p.workers > u0 ? 0 : 1;
  return a.part + ((static_cast<long long>(phase) * ctas + w) * 2 + slot) *
                      (2ll * a.part_tokens * 128);
}

__device__ __forceinline__ int round_up(int x, int m) { return (x + m - 1) / m * m; }

__device__ __forceinline__ void arrive_release(unsigned int* bar) {
  asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(bar) : "memory");
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

  // after the ring: barriers, then the routing lists
  uint8_t* const tail = base_ptr + static_cast<size_t>(S) * a.stage_bytes;
  const uint32_t bars = base + static_cast<uint32_t>(S * a.stage_bytes);
  auto full_bar = [&](int s) { return bars + 8u * s; };                     // weights landed
  auto tok_bar = [&](int s) { return bars + 8u * (kMaxStages + s); };       // token rows staged
  auto empty_bar = [&](int s) { return bars + 8u * (2 * kMaxStages + s); };
  auto accf_bar = [&](uint32_t b) { return bars + 8u * (3 * kMaxStages + b); };
  auto acce_bar = [&](uint32_t b) { return bars + 8u * (3 * kMaxStages + 2 + b); };
  const uint32_t done_bar = bars + 8u * (3 * kMaxStages + 4);
  constexpr int kBarBytes = 8 * (3 * kMaxStages + 5);
  uint32_t* const misc = reinterpret_cast<uint32_t*>(tail + kBarBytes);     // TMEM address, active
  uint16_t* const s_ids = reinterpret_cast<uint16_t*>(tail + kBarBytes + 8);   // expert of a pair
  const int P2 = round_up(P, 2), E2 = round_up(a.E, 2);
  uint16_t* const s_list = s_ids + P2;    // pairs by (expert, pair)
  uint16_t* const s_pos = s_list + P2;    // place of a pair in s_list
  uint16_t* const s_cnt = s_pos + P2;     // tokens of expert e
  uint16_t* const s_off = s_cnt + E2;     // first place of expert e
  uint16_t* const s_qi = s_off + E2;      // rank of expert e among the active ones
  uint16_t* const s_act = s_qi + E2;      // active experts in order

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1u);
      mbar_init(tok_bar(s), 1u);
      mbar_init(empty_bar(s), 1u);
    }
    for (uint32_t b = 0; b < 2; ++b) {
      mbar_init(accf_bar(b), 1u);
      mbar_init(acce_bar(b), static_cast<uint32_t>(kEpi));
    }
    mbar_init(done_bar, 1u);
    fence_barrier_init();
    fence_proxy_async_smem();
    prefetch_tensormap(&tm1);
    prefetch_tensormap(&tm2);
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(misc), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(misc);
  griddep_wait();   // the routing kernel's ids, p and zeroed counters

  // ---- lists: for every expert its pairs in order
  for (int i = threadIdx.x; i < P2; i += kStreamThreads)
    s_ids[i] = i < P ? static_cast<uint16_t>(__ldcg(a.ids + i)) : static_cast<uint16_t>(0xFFFFu);
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kStreamThreads) {
    const uint32_t key = static_cast<uint32_t>(e) * 0x10001u;
    uint32_t n = 0;
    const uint32_t* w = reinterpret_cast<const uint32_t*>(s_ids);
    for (int i = 0; i < P2 / 2; ++i) n += __popc(__vcmpeq2(w[i], key));
    s_cnt[e] = static_cast<uint16_t>(n / 16);
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
        if (n > 0) {
          const int q = act + __popc(some & ((1u << lane) - 1u));
          s_qi[e] = static_cast<uint16_t>(q);
          s_act[q] = static_cast<uint16_t>(e);
        }
      }
      off += __shfl_sync(0xffffffffu, incl, 31);
      act += __popc(some);
    }
    if (lane == 0) misc[1] = static_cast<uint32_t>(act);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kStreamThreads) {
    int left = s_cnt[e], pos = s_off[e];
    for (int i = 0; left > 0; ++i)
      if (s_ids[i] == e) {
        s_list[pos] = static_cast<uint16_t>(i);
        s_pos[i] = static_cast<uint16_t>(pos);
        ++pos;
        --left;
      }
  }
  __syncthreads();
  const int active = static_cast<int>(misc[1]);
  const Phase up = phase_of(active, a.up_tiles, a.up_kb, cta, ctas);
  const Phase down = phase_of(active, a.down_tiles, a.down_kb, cta, ctas);
  const unsigned long long limit = a.wait_limit_ns;
  DeviceStatus* const st = a.status;
  const unsigned int arrivals = static_cast<unsigned int>(kEpi * ctas);

  if (warp == 0) {
    // ---------------------------------------------------------- weights (TMA)
    if (lane == 0) {
      const uint64_t policy = l2_evict_first_policy();
      int stage = 0;
      uint32_t phase = 0, issued = 0;
      bool ok = true;
      for (int ph = 0; ph < 2 && ok; ++ph) {
        const Phase& p = ph ? down : up;
        for (long long x = p.beg; x < p.end && ok;) {
          const Piece t = piece_at(p, x);
          const int e = s_act[t.q];
          // columns of the four boxes; one that lies past the matrix is skipped
          int col[4], n = 0;
          bool use[4];
          for (int b = 0; b < 4; ++b) {
            if (ph == 0) {
              const int j = t.tile * 128 + (b & 1) * 64;
              use[b] = j < a.I;
              col[b] = (b >> 1) * a.I + j;
            } else {
              col[b] = t.tile * 256 + b * 64;
              use[b] = col[b] < a.H;
            }
            n += use[b];
          }
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
                tma_load_3d_hint(dst + b * 8192, ph ? &tm2 : &tm1, full_bar(stage), col[b],
                                 kb * 64, e, policy);
            ++issued;
            if (++stage == S) {
              stage = 0;
              phase ^= 1u;
            }
          }
          x += t.kb1 - t.kb0;
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
      for (int ph = 0; ph < 2 && ok; ++ph) {
        const Phase& p = ph ? down : up;
        for (long long x = p.beg; x < p.end && ok;) {
          const Piece t = piece_at(p, x);
          const int n = s_cnt[s_act[t.q]];
          const int cols = ph ? 2 * round_up(n, 8) : round_up(n, 16);
          const uint32_t idesc = make_idesc(0u, 128u, static_cast<uint32_t>(cols), 1u, 0u);
          const uint32_t buf = local & 1u;
          if (!wait_parity(acce_bar(buf), ((local >> 1) & 1u) ^ 1u, limit, st, 42)) {
            ok = false;
            break;
          }
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
          ++local;
          x += t.kb1 - t.kb0;
        }
      }
      mma_commit(done_bar);
      settle_wait(done_bar, 0u, st, 45);
    }
    __syncwarp();
  } else if (warp < 2 + kLoaders) {
    // ---------------------------------------------------------- token rows
    // Loader l stages the k-blocks l, l + 4, ... of the CTA's sequence: rows
    // of X for up; for down the hi rows of hid, then (from the next multiple
    // of 8) the lo rows.  Rows past them are left as they are: their columns
    // of the product are never read.
    const int l = warp - 2;
    int stage = 0, seq = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int ph = 0; ph < 2 && ok; ++ph) {
      if (ph == 1) {
        // hid of every pair is written (by all CTAs)
        if (lane == 0) ok = wait_count(a.bars, arrivals, limit, st, 46);
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        if (!ok) break;
      }
      const Phase& p = ph ? down : up;
      const int K = ph ? a.I : a.H;
      for (long long x = p.beg; x < p.end && ok;) {
        const Piece t = piece_at(p, x);
        const int e = s_act[t.q];
        const int n = s_cnt[e], off = s_off[e], n8 = round_up(n, 8);
        const int rows = ph ? 2 * n : n;
        for (int kb = t.kb0; kb < t.kb1; ++kb, ++seq) {
          if ((seq & (kLoaders - 1)) == l) {
            if (!wait_parity(empty_bar(stage), phase ^ 1u, limit, st, 47)) {
              ok = false;
              break;
            }
            uint8_t* const dst = base_ptr + static_cast<size_t>(stage) * a.stage_bytes + kWeightBytes;
            for (int i0 = 0; i0 < rows * 8; i0 += 32 * 4) {
              uint4 v[4];
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const int i = i0 + 32 * u + lane;
                const int r = i >> 3, k = kb * 64 + (i & 7) * 8;
                v[u] = make_uint4(0u, 0u, 0u, 0u);
                if (r < rows && k < K) {
                  if (ph == 0) {
                    v[u] = __ldg(reinterpret_cast<const uint4*>(
                        a.X + static_cast<long long>(s_list[off + r] / a.topk) * a.ldx + k));
                  } else {
                    const long long row = off + (r < n ? r : r - n + P);
                    v[u] = __ldcg(reinterpret_cast<const uint4*>(a.hid + row * a.I + k));
                  }
                }
              }
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const int i = i0 + 32 * u + lane;
                const int r = i >> 3, c = i & 7;
                if (r < rows) {
                  const int rr = (ph && r >= n) ? r - n + n8 : r;
                  *reinterpret_cast<uint4*>(dst + rr * 128 + ((c ^ (rr & 7)) << 4)) = v[u];
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
        x += t.kb1 - t.kb0;
      }
    }
  } else {
    // ---------------------------------------------------------- epilogue
    const int quad = warp & 3;                 // TMEM lanes 32 quad ..
    const int col = 32 * quad + lane;          // this thread's column of a 128-wide accumulator
    uint32_t local = 0;
    bool ok = true;
    for (int ph = 0; ph < 2 && ok; ++ph) {
      const Phase& p = ph ? down : up;
      for (long long x = p.beg; x < p.end;) {
        const Piece t = piece_at(p, x);
        const int e = s_act[t.q];
        const int n = s_cnt[e], off = s_off[e], n8 = round_up(n, 8);
        const uint32_t buf = local & 1u;
        if (!wait_parity(accf_bar(buf), (local >> 1) & 1u, limit, st, 48)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d0 =
            tmem + (static_cast<uint32_t>(32 * quad) << 16) + buf * (2 * kAccCols);
        const bool whole = t.kb0 == 0 && t.kb1 == p.kb;
        const long long u0 = t.unit * p.kb;
        // one chunk of 8 tokens of accumulator `acc`, hi and lo parts added
        auto load8 = [&](int r0, float (&v0)[8], float (&v1)[8]) {
          uint32_t g[8], h[8];
          tmem_ld_32x32b_x8(d0 + r0, g);
          tmem_ld_32x32b_x8(d0 + kAccCols + r0, h);
          tmem_wait_ld2(g, h);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            v0[i] = __uint_as_float(g[i]);
            v1[i] = __uint_as_float(h[i]);
          }
          if (ph == 1) {
            tmem_ld_32x32b_x8(d0 + n8 + r0, g);
            tmem_ld_32x32b_x8(d0 + kAccCols + n8 + r0, h);
            tmem_wait_ld2(g, h);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              v0[i] += __uint_as_float(g[i]);
              v1[i] += __uint_as_float(h[i]);
            }
          }
        };
        // hid of 8 tokens at column j
        const int j = t.tile * 128 + col;
        auto store_hid = [&](int r0, const float (&g)[8], const float (&u)[8]) {
          if (j >= a.I) return;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (r0 + i < n) {
              const float h = g[i] / (1.0f + expf(-g[i])) * u[i];
              const uint16_t hi = moe_f2h(h);
              const float rest = h - moe_h2f(hi);
              // past the half range hi is infinite and stands alone
              const uint16_t lo = (hi & 0x7FFFu) >= 0x7C00u ? 0 : moe_f2h(rest);
              const long long o = static_cast<long long>(off + r0 + i) * a.I + j;
              a.hid[o] = hi;
              a.hid[static_cast<long long>(P) * a.I + o] = lo;
            }
        };
        if (whole) {
          for (int r0 = 0; r0 < n; r0 += 8) {
            float v0[8], v1[8];
            load8(r0, v0, v1);
            if (ph == 0) {
              store_hid(r0, v0, v1);
            } else {
              const int c0 = t.tile * 256 + col;
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (r0 + i < n) {
                  float* o = a.z + static_cast<long long>(off + r0 + i) * a.H;
                  if (c0 < a.H) __stcg(o + c0, v0[i]);
                  if (c0 + 128 < a.H) __stcg(o + c0 + 128, v1[i]);
                }
            }
          }
        } else {
          float* const mine = part_of(a, p, ph, cta, ctas, u0) + col;
          for (int r0 = 0; r0 < n; r0 += 8) {
            float v0[8], v1[8];
            load8(r0, v0, v1);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (r0 + i < n) {
                __stcg(mine + (r0 + i) * 128, v0[i]);
                __stcg(mine + (a.part_tokens + r0 + i) * 128, v1[i]);
              }
          }
          if (ph == 0) {
            // the last of the unit's pieces to arrive adds them up in k order
            const int c0 = owner_of(p, u0), c1 = owner_of(p, u0 + p.kb - 1);
            __threadfence();
            __syncwarp();
            unsigned int before = 0;
            if (lane == 0) before = atomicAdd(a.counters + t.unit * kEpi + quad, 1u);
            before = __shfl_sync(0xffffffffu, before, 0);
            if (before == static_cast<unsigned int>(c1 - c0)) {
              __threadfence();
              for (int r0 = 0; r0 < n; r0 += 8) {
                float v0[8] = {}, v1[8] = {};
                for (int w = c0; w <= c1; ++w) {
                  const float* src = part_of(a, p, ph, w, ctas, u0) + col;
#pragma unroll
                  for (int i = 0; i < 8; ++i)
                    if (r0 + i < n) {
                      v0[i] += __ldcg(src + (r0 + i) * 128);
                      v1[i] += __ldcg(src + (a.part_tokens + r0 + i) * 128);
                    }
                }
                store_hid(r0, v0, v1);
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acce_bar(buf));
        ++local;
        x += t.kb1 - t.kb0;
      }
      // this warp's share of the phase is written
      __threadfence();
      __syncwarp();
      if (ok && lane == 0) arrive_release(a.bars + ph);
    }
  }

  // ---- sum: z of every pair is written; a warp per (token, 32 columns)
  bool ready = true;
  if (lane == 0) ready = wait_count(a.bars + 1, arrivals, limit, st, 49);
  ready = __shfl_sync(0xffffffffu, ready ? 1 : 0, 0) != 0;
  if (ready) {
    const int strips = (a.H + 31) / 32;
    for (int it = cta * kStreamWarps + warp; it < a.T * strips; it += ctas * kStreamWarps) {
      const int t = it / strips, c = (it - t * strips) * 32 + lane;
      const int tile = (it - t * strips) / 8;          // 256-column tile, uniform in the warp
      const int in_tile = c - tile * 256;              // 0 .. 255
      float y = 0.0f;
      for (int k = 0; k < a.topk; ++k) {
        const int pair = t * a.topk + k, e = s_ids[pair], pos = s_pos[pair];
        const long long u0 = (static_cast<long long>(s_qi[e]) * a.down_tiles + tile) * a.down_kb;
        const int c0 = owner_of(down, u0), c1 = owner_of(down, u0 + a.down_kb - 1);
        float z = 0.0f;
        if (c0 == c1) {
          if (c < a.H) z = __ldcg(a.z + static_cast<long long>(pos) * a.H + c);
        } else {
          const int r = pos - s_off[e];
          for (int w = c0; w <= c1; ++w)
            z += __ldcg(part_of(a, down, 1, w, ctas, u0) +
                        ((in_tile >> 7) * a.part_tokens + r) * 128 + (in_tile & 127));
        }
        y = fmaf(__ldcg(a.probs + pair), z, y);
      }
      if (c < a.H) {
        uint16_t* o = a.Y + static_cast<long long>(t) * a.ldy + c;
        *o = moe_f2h(a.beta != 0.0f ? fmaf(a.beta, moe_h2f(*o), y) : y);
      }
    }
  }
  __syncthreads();   // the epilogue warps have read TMEM, the MMAs are complete
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

bool moe_stream_fits(const MoeArgs& m) {
  const uintptr_t ptrs = reinterpret_cast<uintptr_t>(m.X) | reinterpret_cast<uintptr_t>(m.W1) |
                         reinterpret_cast<uintptr_t>(m.W2);
  // the rows of X, W1 (2I halves) and W2 (H) on the 16-byte grid
  return (ptrs & 15u) == 0 && m.H % 8 == 0 && m.I % 8 == 0 && m.ldx % 8 == 0 && m.I > 0;
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
    s.part_tokens = T;
    s.wait_limit_ns = limit_ns;
    s.status = st;
    // token rows of a stage: X rows padded to 16, or hi and lo rows padded to 8
    const int rows = std::max((T + 15) / 16 * 16, 2 * ((T + 7) / 8 * 8));
    s.stage_bytes = kWeightBytes + rows * 128;
    const int lists = 8 * (3 * kMaxStages + 5) + 8 + 2 * (3 * (P + 1) + 4 * (m.E + 1));
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
    const int want = std::max(1, std::min({sms / (r.egroups * r.tblocks), 16, m.H / 32}));
    r.rows_per_split = (m.H + want - 1) / want;
    r.splits = (m.H + r.rows_per_split - 1) / r.rows_per_split;

    const long long units = 1ll * std::min(m.E, P) * s.up_tiles;
    const size_t b_part = round256(4 * static_cast<size_t>(r.splits) * T * m.E);
    const size_t b_ids = round256(4 * static_cast<size_t>(P));
    const size_t b_hid = round256(2 * 2 * static_cast<size_t>(P) * m.I);
    const size_t b_z = round256(4 * static_cast<size_t>(P) * m.H);
    const size_t b_ws = round256(4 * 2 * static_cast<size_t>(sms) * 2 * 2 * T * 128);
    const size_t b_cnt = round256(4 * (static_cast<size_t>(units) * kEpi + 2));
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
    s.hid = reinterpret_cast<uint16_t*>(take(b_hid));
    s.z = reinterpret_cast<float*>(take(b_z));
    s.part = reinterpret_cast<float*>(take(b_ws));
    s.bars = reinterpret_cast<unsigned int*>(take(b_cnt));
    s.counters = s.bars + 2;
    s.ids = r.ids;
    s.probs = r.probs;
    r.counters = static_cast<unsigned int*>(zero);
    r.zero = s.bars;
    r.nzero = static_cast<int>(units * kEpi + 2);
    r.ids_out = m.ids ? m.ids + static_cast<long long>(t0) * m.topk : nullptr;
    r.probs_out = m.probs ? m.probs + static_cast<long long>(t0) * m.topk : nullptr;

    const size_t route_smem = static_cast<size_t>(kRouteT) * m.E * 5;
    moe_logits_kernel<<<r.tblocks * r.egroups * r.splits, kRouteThreads, route_smem, stream>>>(r);
    if (counted_launch(cudaGetLastError()) != cudaSuccess) return GEMM_ERR_CUDA;

    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(sms), 1, 1);
    cfg.blockDim = dim3(kStreamThreads, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(s.stages) * s.stage_bytes + lists + 1024;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
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
