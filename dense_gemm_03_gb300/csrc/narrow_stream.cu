// narrow_stream.cu -- products of halves with few rows or few tiles: W is the M operand
// of tcgen05.mma (128 of its columns), the rows of X the N operand, K is cut into chunks
// that go to different SMs.
//
// Two ways to add the chunks up:
//   cluster    as many chunks as a cluster has CTAs (1, 2, 4 or 8), each CTA one chunk of
//              one tile; the sums meet in shared memory, each CTA adds up its share of the
//              outputs through distributed shared memory, finishes and stores them.  One
//              launch, no partial sums in global memory: for products that one wave
//              of CTAs covers
//   partial    fp32 partial sums of any number of chunks over persistent CTAs, added up
//              by stream_sum.cu: for W that takes longer than that, where evenly shared
//              work counts for more
// A gate's unit is 64 of its columns and the 64 that they gate, so that a CTA of the cluster
// form has both sums of an output.
//
// Steps are 128 deep, and a step's tile of W (and of X) is one TMA instruction where
// the sizes allow (maps of three dimensions): the thread that issues them takes about
// 0.1 us for each, so that with 64-deep steps of three instructions a CTA took in 16 KB of
// W in 0.31 us, whatever the bytes.  The first loads are issued before tensor memory is
// allocated and the CTA's threads have met.
//
// What bounds: one token of 2048 x 2*4096, 34 MB of W, takes 8.4 us: 4.6 us at the HBM rate
// and the chain of a launch, the first load's latency and two cluster barriers.
//
// Shared memory: ring stages of W, two 64-column blocks [128 k][64 halves]
// (MN-major, 128-byte swizzle, LBO 16 KB), or of a W stored transposed two 64-deep blocks
// [128 columns][64 halves] (K-major); then X, two 64-deep blocks [row][64 halves]
// (K-major), or 64-row blocks [128 k][64 halves].
#include "narrow.cuh"

namespace gb300 {
namespace {

constexpr int kWBytes = kStepK * 256;       // 128 columns of a step
constexpr int kMaxStages = 8;
constexpr int kEpi = 8;                     // warps that write sums
constexpr int kThreads = 64 + 32 * kEpi;
constexpr int kBlockRows = 256;

struct Args : Tiles {
  int stages, stage_bytes, x_bytes, bar_off;
  bool trans_w, trans_x;
  bool one_w, one_x;            // the step's tile is one instruction
};

template <int FIN>
__global__ void __launch_bounds__(kThreads, 1)
    narrow_stream_kernel(const __grid_constant__ CUtensorMap tmW,
                         const __grid_constant__ CUtensorMap tmX, const Args p, const StreamSum fin) {
  constexpr bool kCluster = FIN != kPartial;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw0 = smem_addr(smem_raw);
  const uint32_t base = (raw0 + 1023u) & ~1023u;
  uint8_t* const base_ptr = smem_raw + (base - raw0);
  const int S = p.stages;
  const int warp = warp_id_uniform(), lane = static_cast<int>(lane_id());
  const uint32_t bars = base + static_cast<uint32_t>(p.bar_off);
  auto full_bar = [&](int s) { return bars + 8u * s; };
  auto empty_bar = [&](int s) { return bars + 8u * (kMaxStages + s); };
  const uint32_t acc_full = bars + 8u * (2 * kMaxStages);
  const uint32_t acc_empty = acc_full + 8u, done_bar = acc_full + 16u;
  uint8_t* const tmem_ptr = base_ptr + p.bar_off + 8 * (2 * kMaxStages + 3);
  const unsigned long long limit = p.wait_limit_ns;
  DeviceStatus* const st = p.status;
  // one step's loads into stage s
  const uint64_t policy = l2_evict_first_policy();
  auto load_step = [&](int s, int n0, int row0, int step) {
    const uint32_t dst = base + static_cast<uint32_t>(s * p.stage_bytes), bar = full_bar(s);
    const int k = step * kStepK;
    mbar_arrive_expect_tx(bar, static_cast<uint32_t>(p.stage_bytes));
    // W, evict-first when no other block of rows reads it
    auto w2 = [&](uint32_t to, int cx, int cy) {
      if (p.reread)
        tma_load_2d(to, &tmW, bar, cx, cy);
      else
        tma_load_2d_hint(to, &tmW, bar, cx, cy, policy);
    };
    auto w3 = [&](int cx, int cy, int cz) {
      if (p.reread)
        tma_load_3d(dst, &tmW, bar, cx, cy, cz);
      else
        tma_load_3d_hint(dst, &tmW, bar, cx, cy, cz, policy);
    };
    if (p.trans_w) {
      if (p.one_w) {
        w3(0, n0, 2 * step);       // [64 k][column][k]
      } else {
        w2(dst, k, n0);
        w2(dst + kWBytes / 2, k + 64, n0);
      }
    } else if (p.one_w) {
      if (paired<FIN>())
        w3(n0, k, 0);              // [gate or up][k][column]
      else
        w3(0, k, n0 / 64);         // [64 columns][k][column]
    } else {
      w2(dst, n0, k);
      w2(dst + kWBytes / 2, n0 + 64, k);
    }
    const uint32_t x = dst + kWBytes;
    if (p.trans_x) {
      if (p.one_x)
        tma_load_3d(x, &tmX, bar, 0, k, row0 / 64);   // [64 rows][k][row]
      else
        for (int b = 0; b < p.x_bytes; b += 16384) tma_load_2d(x + b, &tmX, bar, row0 + b / 256, k);
    } else if (p.one_x) {
      tma_load_3d(x, &tmX, bar, 0, row0, 2 * step);   // [64 k][row][k]
    } else {
      tma_load_2d(x, &tmX, bar, k, row0);
      tma_load_2d(x + p.x_bytes / 2, &tmX, bar, k + 64, row0);
    }
  };
  if (warp == 0) {
    // barriers, a lane each
    if (lane < S) {
      mbar_init(full_bar(lane), 1u);
      mbar_init(empty_bar(lane), 1u);
    }
    if (lane == 31) {
      mbar_init(acc_full, 1u);
      mbar_init(acc_empty, static_cast<uint32_t>(kEpi));
      mbar_init(done_bar, 1u);
    }
    fence_barrier_init();
    fence_proxy_async_smem();
    __syncwarp();
    if (!p.beside) griddep_wait();   // copies onto the 16-byte grid, if any
    // the first item's first steps: their stages are empty
    if (lane == 0) {
      const int it = blockIdx.x, n = min(S, p.steps(it));
      for (int s = 0; s < n; ++s) load_step(s, p.n0(it), p.row0(it), p.first_step(it) + s);
    }
    __syncwarp();
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(tmem_ptr), p.acc_cols);
    tmem_relinquish();
    griddep_launch_dependents();   // only now: see lora_stream.cu
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp > 0 && !p.beside) griddep_wait();   // (what the results are joined with)
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_ptr);

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      // (the first item's first steps are on their way)
      int skip = min(S, p.steps(blockIdx.x)), s = 0;
      uint32_t phase = 0, issued = 0;
      bool ok = true;
      for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
        const int n0 = p.n0(it), row0 = p.row0(it), end = p.first_step(it) + p.steps(it);
        for (int step = p.first_step(it); step < end; ++step) {
          if (skip > 0) {
            --skip;
          } else {
            if (!wait_parity(empty_bar(s), phase ^ 1u, limit, st, 70)) {
              ok = false;
              break;
            }
            load_step(s, n0, row0, step);
          }
          ++issued;
          if (++s == S) {
            s = 0;
            phase ^= 1u;
          }
        }
      }
      const uint32_t n = min(issued, static_cast<uint32_t>(S));
      for (uint32_t i = issued - n; i < issued; ++i)
        settle_wait(full_bar(static_cast<int>(i % S)), (i / S) & 1u, st, 71);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      const uint32_t idesc = make_idesc(0u, 128u, static_cast<uint32_t>(p.n_cols),
                                        p.trans_w ? 0u : 1u, p.trans_x ? 1u : 0u);
      // The loop of this one thread can set the pace: descriptors are added up, not
      // built, and the next step's barrier is looked at before this step's MMAs.
      const uint32_t stride = static_cast<uint32_t>(p.stage_bytes) >> 4;
      const bool tw = p.trans_w, tx = p.trans_x;
      const uint64_t wd0 = smem_desc_sw128(base, tw ? 16u : 16384u, 1024u);
      const uint64_t xd0 = smem_desc_sw128(base + kWBytes, tx ? 16384u : 16u, 1024u);
      // 16 k and 64 k on, in 16 bytes
      const uint32_t wk = tw ? 2u : 128u, wq = tw ? 1024u : 512u;
      const uint32_t xk = tx ? 128u : 2u, xq = tx ? 512u : static_cast<uint32_t>(p.n_cols) * 8u;
      int s = 0;
      uint32_t phase = 0, local = 0, off = 0;
      bool ok = true, ready = false;
      for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x, ++local) {
        int left = p.steps(it);
        if (!wait_parity(acc_empty, (local & 1u) ^ 1u, limit, st, 72)) break;
        tc_fence_after();
        for (uint32_t acc = 0; left > 0; --left) {
          if (!ready && !wait_parity(full_bar(s), phase, limit, st, 73)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t done = empty_bar(s);
          const uint64_t wd = wd0 + off, xd = xd0 + off;
          off += stride;
          if (++s == S) {
            s = 0;
            off = 0;
            phase ^= 1u;
          }
          ready = left > 1 && mbar_test_wait(full_bar(s), phase);
#pragma unroll
          for (uint32_t kk = 0; kk < 8; ++kk) {
            mma_f16_ss(tmem, wd + ((kk >> 2) * wq + (kk & 3) * wk), xd + ((kk >> 2) * xq + (kk & 3) * xk),
                       idesc, acc);
            acc = 1u;
          }
          mma_commit(done);
        }
        if (!ok) break;
        mma_commit(acc_full);
      }
      mma_commit(done_bar);
      settle_wait(done_bar, 0u, st, 74);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ sums
    const int quad = warp & 3, part = (warp - 2) >> 2;
    uint32_t local = 0;
    for (int it = blockIdx.x; it < p.items; it += gridDim.x, ++local) {
      if (!wait_parity(acc_full, local & 1u, limit, st, 77)) break;
      tc_fence_after();
      // to global memory or, the ring being done with, to the start of shared memory
      write_sums(tmem, 0u, quad, lane, part, kEpi / 4, min(p.rows, p.M - p.row0(it)),
                 kCluster ? reinterpret_cast<float*>(base_ptr)
                          : p.part + static_cast<long long>(it) * p.rows * 128);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty);
    }
  }
  if constexpr (kCluster)
    cluster_finish<FIN>(p, fin, base, kThreads);
  else
    __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, p.acc_cols);
  if (p.beside && blockIdx.x + 1 == gridDim.x) griddep_wait();   // the grid ends no sooner
}

// Stages and the place of the barriers, for `steps` steps a CTA at most.
void lay_out(Args& a, const NarrowStream& p, int steps, bool cluster) {
  a.trans_w = p.trans_w;
  a.beside = p.beside;
  a.trans_x = p.trans_x;
  a.x_bytes = a.trans_x ? (a.n_cols + 63) / 64 * 16384 : a.n_cols * 256;
  a.stage_bytes = kWBytes + a.x_bytes;
  a.stages = std::min({kMaxStages, (kSmemMax - 2048) / a.stage_bytes, steps});
  a.bar_off = std::max(a.stages * a.stage_bytes, cluster ? a.n_cols * 512 : 0);
}

template <int FIN>
int launch(const Args& a, const StreamSum& fin, const CUtensorMap& tmW, const CUtensorMap& tmX,
           int grid, cudaStream_t stream) {
  static bool configured[64] = {};
  return launch_narrow(narrow_stream_kernel<FIN>, kThreads, static_cast<size_t>(a.bar_off) + 2048,
                       grid, FIN == kPartial ? 0 : a.chunks, configured, stream, tmW, tmX, a,
                       fin);
}

// The maps of the operands.  Three dimensions, so that a step is one instruction,
// where they stay inside the matrix: 64-column (or 64-row, 64-deep) blocks as the third
// dimension of one whose size is a multiple of 64; a gate's columns and those it
// gates.  `paired`: the latter, U's columns `up` after G's.
int make_maps(Args& a, const NarrowStream& p, bool paired, int up, CUtensorMap* tmW,
              CUtensorMap* tmX) {
  const int K = p.K;
  int rc;
  if (a.trans_w) {
    a.one_w = K % 64 == 0;
    rc = a.one_w ? encode_map_3d(tmW, 2, p.W, {64, a.N, K / 64}, {p.ldw, 64}, {64, 128, 2})
                 : encode_map_3d(tmW, 2, p.W, {K, a.N, 0}, {p.ldw, 0}, {64, 128, 0});
  } else if (paired) {
    a.one_w = true;
    rc = encode_map_3d(tmW, 2, p.W, {up, K, 2}, {p.ldw, up}, {64, kStepK, 2});
  } else {
    a.one_w = a.N % 64 == 0;
    rc = a.one_w ? encode_map_3d(tmW, 2, p.W, {64, K, a.N / 64}, {p.ldw, 64}, {64, kStepK, 2})
                 : encode_map_3d(tmW, 2, p.W, {a.N, K, 0}, {p.ldw, 0}, {64, kStepK, 0});
  }
  if (rc) return rc;
  if (a.trans_x) {
    a.one_x = block_of_64s(a.M, a.rows);   // (its coordinate counts 64-row blocks)
    return a.one_x ? encode_map_3d(tmX, 2, p.X, {64, K, a.M / 64}, {p.ldx, 64},
                                   {64, kStepK, (a.n_cols + 63) / 64})
                   : encode_map_3d(tmX, 2, p.X, {a.M, K, 0}, {p.ldx, 0}, {64, kStepK, 0});
  }
  a.one_x = K % 64 == 0;
  return a.one_x ? encode_map_3d(tmX, 2, p.X, {64, a.M, K / 64}, {p.ldx, 64}, {64, a.n_cols, 2})
                 : encode_map_3d(tmX, 2, p.X, {K, a.M, 0}, {p.ldx, 0}, {64, a.n_cols, 0});
}

// The longest of `chunks` chunks of K.
int longest_chunk(int K, int chunks) {
  const int steps = (K + kStepK - 1) / kStepK;
  return std::min(K, (steps + chunks - 1) / chunks * kStepK);
}

Args plan_partial(const NarrowStream& p, int M, int cols, bool fold, const LoraDevice& d) {
  Args a{};
  // chunks of kFoldDepth at most
  const int least = fold ? ((p.K + kStepK - 1) / kStepK - 1) / (kFoldDepth / kStepK) + 1 : 1;
  static_cast<Tiles&>(a) = partial_tiles(M, cols, p.K, kBlockRows, p.trans_x, (p.K + 63) / 64, least, d);
  lay_out(a, p, kMaxStages, false);
  return a;
}

}  // namespace

StreamParts narrow_parts(const NarrowStream& p, int M, int cols, bool fold, const LoraDevice& d) {
  const Args a = plan_partial(p, M, cols, fold, d);
  return StreamParts{nullptr, a.chunks, a.units, a.rows,
                     4 * static_cast<size_t>(a.items) * a.rows * 128, a.rows};
}

int narrow_partial(const NarrowStream& p, int M, int cols, bool fold, const StreamParts& parts,
                   const LoraDevice& d, cudaStream_t stream) {
  Args a = plan_partial(p, M, cols, fold, d);
  a.part = parts.part;
  CUtensorMap tmW{}, tmX{};
  if (int rc = make_maps(a, p, false, 0, &tmW, &tmX)) return rc;
  return launch<kPartial>(a, StreamSum{}, tmW, tmX, std::min(a.items, d.sms), stream);
}

bool narrow_cluster_suits(const NarrowStream& p, const StreamSum& s, const LoraDevice& d) {
  if (s.gate && s.N % 8 != 0) return false;   // U's columns start on TMA's 16-byte grid
  const Tiles a = cluster_tiles(s, p.K, kBlockRows, p.trans_x, d);
  return cluster_pays(a, d.sms) && (!(s.f32 || s.fold) || longest_chunk(p.K, a.chunks) <= kFoldDepth);
}

int narrow_cluster(const NarrowStream& p, const StreamSum& s, const LoraDevice& d,
                   cudaStream_t stream) {
  Args a{};
  static_cast<Tiles&>(a) = cluster_tiles(s, p.K, kBlockRows, p.trans_x, d);
  if (a.chunks == 0) return GEMM_ERR_ARG;
  lay_out(a, p, (a.kb + a.chunks - 1) / a.chunks, true);
  CUtensorMap tmW{}, tmX{};
  if (int rc = make_maps(a, p, s.gate != 0, s.N, &tmW, &tmX)) return rc;
  return s.gate == 2 ? launch<kGateGrad>(a, s, tmW, tmX, a.items, stream)
         : s.gate    ? launch<kGate>(a, s, tmW, tmX, a.items, stream)
         : s.f32     ? launch<kFloat>(a, s, tmW, tmX, a.items, stream)
                     : launch<kHalf>(a, s, tmW, tmX, a.items, stream);
}

}  // namespace gb300
