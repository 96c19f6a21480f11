// i8_stream.cu -- products in 8-bit integers with few rows or few tiles, cut like those
// of halves (narrow_stream.cu): clusters whose sums meet, or partial sums.
//
// This card's tensor cores run 8-bit integers far below halves, and every 8-bit integer
// is a half exactly: W and X come from HBM as bytes by TMA and become halves on their way
// to the tensor cores.  Products are exact, and so are the fp32 sums while they stay
// below 2^24 (always for K <= 1024).
//
// W, K x N with its columns neighbours, is to be the M operand of tcgen05.mma, a column to a
// lane of tensor memory.  ldmatrix transposes 16 x 16 bytes: thread 4 g + t gets bytes k =
// 4 t .. 4 t + 3 of column g, which become two pairs of halves, and those are what
// tcgen05.st takes for lane g, columns t and 4 + t of eight.  So slot 2 t (8 + 2 t) of 16 k
// holds k = 4 t (4 t + 2); the pieces of X are put into the same order.  W as halves
// never touches shared memory: as an operand there it was 32 KB to write and 32 KB to
// read for each 16 KB that came in, which, with the 32 KB on the way to the
// registers, took a CTA 0.59 us a step.  (Loaded into registers from global memory without TMA it was
// 1.1 us: the loads that were to run ahead did not.)
//
// Warps: 16 convert (quadrant q = warp % 4 has lanes, columns of W, 32 q .. + 31; warp / 4
// the 32 k of the step), then write the sums; two issue the MMAs, one the loads.
//
// Shared memory: kBufs buffers of X as halves, two 64-deep halves [row][64 halves]
// (K-major, 128-byte swizzle); then ring stages of raw steps, W as [128 k][128 bytes]
// (of a gate, in the cluster form, two blocks [128 k][64 bytes]) and X as [row][128
// bytes], swizzled over their rows.  Tensor memory: the issuers' sums, 128 columns each,
// then kBufs buffers of 64 columns of W.
#include "i8_convert.cuh"
#include "narrow.cuh"
#include "ptx_i8.cuh"

namespace gb300 {
namespace {

constexpr int kRawW = kStepK * 128;         // a step of 128 columns
constexpr int kMaxStages = 8;
constexpr int kBufs = 4;                    // of operands
constexpr int kWarps = 16;                  // converting, then writing sums
constexpr int kIssuers = 2;
constexpr int kMmaWarp = kWarps, kLoadWarp = kWarps + kIssuers;
constexpr int kThreads = 32 * (kWarps + kIssuers + 1);
constexpr int kBlockRows = 128;
constexpr int kTmemW = 128 * kIssuers;      // first column of W's buffers
constexpr int kTmemCols = 512;

struct Args : Tiles {
  int stages, raw_bytes, buf_bytes, bar_off;
};

template <int FIN>
__global__ void __launch_bounds__(kThreads, 1)
    i8_stream_kernel(const __grid_constant__ CUtensorMap tmW,
                     const __grid_constant__ CUtensorMap tmX, const Args p, const StreamSum fin) {
  constexpr bool kCluster = FIN != kPartial;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw0 = smem_addr(smem_raw);
  const uint32_t base = (raw0 + 1023u) & ~1023u;
  uint8_t* const base_ptr = smem_raw + (base - raw0);
  const int S = p.stages;
  const int warp = warp_id_uniform(), lane = static_cast<int>(lane_id());
  const uint32_t raws = base + static_cast<uint32_t>(kBufs * p.buf_bytes);
  const uint32_t bars = base + static_cast<uint32_t>(p.bar_off);
  auto raw_full = [&](int s) { return bars + 8u * s; };
  auto raw_empty = [&](int s) { return bars + 8u * (kMaxStages + s); };
  auto op_full = [&](int b) { return bars + 8u * (2 * kMaxStages + b); };
  auto op_empty = [&](int b) { return bars + 8u * (2 * kMaxStages + kBufs + b); };
  const uint32_t acc_full = bars + 8u * (2 * kMaxStages + 2 * kBufs);
  const uint32_t acc_empty = acc_full + 8u, done_bar = acc_full + 16u;
  uint8_t* const tmem_ptr = base_ptr + p.bar_off + 8 * (2 * kMaxStages + 2 * kBufs + 3);
  const unsigned long long limit = p.wait_limit_ns;
  DeviceStatus* const st = p.status;

  const uint64_t policy = l2_evict_first_policy();
  auto load_step = [&](int s, int n0, int row0, int step) {
    const uint32_t dst = raws + static_cast<uint32_t>(s * p.raw_bytes), bar = raw_full(s);
    const int k = step * kStepK;
    mbar_arrive_expect_tx(bar, static_cast<uint32_t>(p.raw_bytes));
    // W, evict-first when no other block of rows reads it
    if (paired<FIN>()) {   // [gate or up][k][column]
      if (p.reread)
        tma_load_3d(dst, &tmW, bar, n0, k, 0);
      else
        tma_load_3d_hint(dst, &tmW, bar, n0, k, 0, policy);
    } else if (p.reread) {
      tma_load_2d(dst, &tmW, bar, n0, k);
    } else {
      tma_load_2d_hint(dst, &tmW, bar, n0, k, policy);
    }
    tma_load_2d(dst + kRawW, &tmX, bar, k, row0);
  };
  if (warp == kLoadWarp) {
    // barriers, a lane each
    if (lane < S) {
      mbar_init(raw_full(lane), 1u);
      mbar_init(raw_empty(lane), kWarps);
    }
    if (lane < kBufs) {
      mbar_init(op_full(lane), kWarps);
      mbar_init(op_empty(lane), 1u);
    }
    if (lane == 31) {
      mbar_init(acc_full, kIssuers);
      mbar_init(acc_empty, kWarps);
      mbar_init(done_bar, kIssuers);
    }
    fence_barrier_init();
    fence_proxy_async_smem();
    __syncwarp();
    griddep_wait();   // copies onto the 16-byte grid, if any
    // the first item's first steps: their stages are empty
    if (lane == 0) {
      const int it = blockIdx.x, n = min(S, p.steps(it));
      for (int s = 0; s < n; ++s) load_step(s, p.n0(it), p.row0(it), p.first_step(it) + s);
    }
    __syncwarp();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_addr(tmem_ptr), kTmemCols);
    tmem_relinquish();
    griddep_launch_dependents();   // only now: see lora_stream.cu
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp != kLoadWarp) griddep_wait();   // (what the results are joined with)
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_ptr);

  if (warp == kLoadWarp) {
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
            if (!wait_parity(raw_empty(s), phase ^ 1u, limit, st, 70)) {
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
        settle_wait(raw_full(static_cast<int>(i % S)), (i / S) & 1u, st, 71);
    }
    __syncwarp();
  } else if (warp >= kMmaWarp) {
    // ------------------------------------------------------------ MMA issuers
    // Issuer i takes the item's steps i, i + 2, ... into sums of its own: one thread took
    // 0.43 us for a step's eight MMAs, their barriers and the loop, more than HBM for
    // the step.
    if (lane == 0) {
      const int me = warp - kMmaWarp;
      // A (W) K-major in tensor memory, B (X) K-major in shared memory
      const uint32_t idesc = make_idesc(0u, 128u, static_cast<uint32_t>(p.n_cols), 0u, 0u);
      // (descriptors are added up, and the next buffer's barrier is looked at before this
      // one's MMAs: see narrow_stream.cu)
      const uint32_t stride = static_cast<uint32_t>(p.buf_bytes) >> 4;
      const uint64_t xd0 = smem_desc_sw128(base, 16u, 1024u);
      const uint32_t xq = static_cast<uint32_t>(p.n_cols) * 8u;   // 64 k on, in 16 bytes
      uint32_t step = 0, local = 0;   // of all items'
      bool ok = true, ready = false;
      for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x, ++local) {
        const uint32_t end = step + static_cast<uint32_t>(p.steps(it));
        if (!wait_parity(acc_empty, (local & 1u) ^ 1u, limit, st, 72)) break;
        tc_fence_after();
        ready = false;
        for (uint32_t n = step + me, acc = 0; n < end; n += kIssuers) {
          const uint32_t b = n % kBufs, next = n + kIssuers;
          if (!ready && !wait_parity(op_full(b), (n / kBufs) & 1u, limit, st, 73)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t wt = tmem + kTmemW + 64u * b;
          const uint64_t xd = xd0 + b * stride;
          ready = next < end && mbar_test_wait(op_full(next % kBufs), (next / kBufs) & 1u);
#pragma unroll
          for (uint32_t kk = 0; kk < 8; ++kk) {
            mma_f16_ts(tmem + 128u * me, wt + 8u * kk, xd + ((kk >> 2) * xq + (kk & 3) * 2u), idesc,
                       acc);
            acc = 1u;
          }
          mma_commit(op_empty(b));
        }
        step = end;
        if (!ok) break;
        mma_commit(acc_full);
      }
      mma_commit(done_bar);
      settle_wait(done_bar, 0u, st, 74);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ converters, sums
    const int quad = warp & 3, part = warp >> 2, t = static_cast<int>(threadIdx.x);
    // W: this lane's row of the two matrices (k 16 lane / 16 + lane % 16 of the warp's 32),
    // 16 columns 32 quad + 16 m
    const int k = 32 * part + lane;
    auto w_at = [&](int m) {
      const int c = 2 * quad + m;   // 16-byte piece of the step's 128 columns
      return paired<FIN>() ? (c >> 2) * 8192 + k * 64 + (((c & 3) ^ ((k >> 1) & 3)) << 4)
                           : k * 128 + ((c ^ (k & 7)) << 4);
    };
    const int w0 = w_at(0), w1 = w_at(1);
    const uint32_t wt = tmem + (static_cast<uint32_t>(32 * quad) << 16) + kTmemW + 16u * part;
    // X: 16-byte piece c (16 k) of row r; pieces 4 .. 7 store their halves the other way
    // round, so that the eight threads of a row touch all banks
    const int r8 = t >> 3, c8 = t & 7, j = (c8 & 3) * 2;
    const bool second = c8 >= 4;
    const int x_raw = kRawW + r8 * 128 + ((c8 ^ (r8 & 7)) << 4);
    const int x_to = (second ? p.n_cols * 128 : 0) + r8 * 128;
    const int x0 = x_to + (((j + second) ^ (r8 & 7)) << 4);
    const int x1 = x_to + (((j + !second) ^ (r8 & 7)) << 4);
    int s = 0, b = 0;
    uint32_t phase = 0, op_phase = 0, local = 0;
    bool ok = true;
    for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x, ++local) {
      for (int left = p.steps(it); left > 0; --left) {
        if (!wait_parity(raw_full(s), phase, limit, st, 75) ||
            !wait_parity(op_empty(b), op_phase ^ 1u, limit, st, 76)) {
          ok = false;
          break;
        }
        tc_fence_after();   // the MMAs that read this buffer's tensor memory are done
        const uint32_t src = raws + static_cast<uint32_t>(s * p.raw_bytes);
        uint32_t q[2][4];
        ldmatrix_b8_trans_x2(src + w0, q[0]);
        ldmatrix_b8_trans_x2(src + w1, q[1]);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          // of columns g and g + 8 (i), 16 k each (h)
          uint32_t v[8];
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint2 e = i8_halves(q[m][2 * h + i]);
              v[4 * h + i] = e.x;
              v[4 * h + 2 + i] = e.y;
            }
          tmem_st_16x128b_x4(wt + (static_cast<uint32_t>(16 * m) << 16) + 64u * b, v);
        }
        const uint8_t* const raw_ptr = base_ptr + (src - base);
        uint8_t* const op = base_ptr + static_cast<size_t>(b) * p.buf_bytes;
        for (int r = 0; r + r8 < p.n_cols; r += 4 * kWarps) {
          const uint4 x = *reinterpret_cast<const uint4*>(raw_ptr + x_raw + r * 128);
          const uint2 e0 = i8_halves(x.x), e1 = i8_halves(x.y), e2 = i8_halves(x.z),
                      e3 = i8_halves(x.w);
          const uint4 lo = make_uint4(e0.x, e1.x, e2.x, e3.x), hi = make_uint4(e0.y, e1.y, e2.y, e3.y);
          *reinterpret_cast<uint4*>(op + x0 + r * 128) = second ? hi : lo;
          *reinterpret_cast<uint4*>(op + x1 + r * 128) = second ? lo : hi;
        }
        fence_proxy_async_smem();   // generic writes -> tensor-core reads
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(raw_empty(s));
          mbar_arrive(op_full(b));
        }
        if (++s == S) {
          s = 0;
          phase ^= 1u;
        }
        if (++b == kBufs) {
          b = 0;
          op_phase ^= 1u;
        }
      }
      if (!ok || !wait_parity(acc_full, local & 1u, limit, st, 77)) {
        ok = false;
        break;
      }
      tc_fence_after();
      // to global memory or, the buffers being done with, to the start of shared memory
      write_sums(tmem, p.steps(it) > 1 ? 128u : 0u, quad, lane, part,
                 kWarps / 4, min(p.rows, p.M - p.row0(it)),
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
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

void lay_out(Args& a, int steps, bool cluster) {
  a.buf_bytes = a.n_cols * 256;
  a.raw_bytes = kRawW + a.n_cols * 128;
  a.stages = std::min({kMaxStages, (kSmemMax - 2048 - kBufs * a.buf_bytes) / a.raw_bytes, steps});
  a.bar_off = std::max(kBufs * a.buf_bytes + a.stages * a.raw_bytes, cluster ? a.n_cols * 512 : 0);
}

template <int FIN>
int launch(const Args& a, const NarrowStream& p, const StreamSum& fin, int grid,
           cudaStream_t stream) {
  CUtensorMap tmW{}, tmX{};
  if (int rc = paired<FIN>()
                   ? encode_map_3d(&tmW, 1, p.W, {fin.N, p.K, 2}, {p.ldw, fin.N}, {64, kStepK, 2})
                   : encode_map_3d(&tmW, 1, p.W, {a.N, p.K, 0}, {p.ldw, 0}, {128, kStepK, 0}))
    return rc;
  if (int rc = encode_map_3d(&tmX, 1, p.X, {p.K, a.M, 0}, {p.ldx, 0}, {kStepK, a.n_cols, 0}))
    return rc;
  static bool configured[64] = {};
  return launch_narrow(i8_stream_kernel<FIN>, kThreads, static_cast<size_t>(a.bar_off) + 2048, grid,
                       FIN == kPartial ? 0 : a.chunks, configured, stream, tmW, tmX, a, fin);
}

Args plan_partial(const NarrowStream& p, int M, int cols, const LoraDevice& d) {
  Args a{};
  static_cast<Tiles&>(a) = partial_tiles(M, cols, p.K, kBlockRows, false, (p.K + 127) / 128, 1, d);
  lay_out(a, kMaxStages, false);
  return a;
}

}  // namespace

StreamParts i8_parts(const NarrowStream& p, int M, int cols, const LoraDevice& d) {
  const Args a = plan_partial(p, M, cols, d);
  return StreamParts{nullptr, a.chunks, a.units, a.rows,
                     4 * static_cast<size_t>(a.items) * a.rows * 128, a.rows};
}

int i8_partial(const NarrowStream& p, int M, int cols, const StreamParts& parts,
               const LoraDevice& d, cudaStream_t stream) {
  Args a = plan_partial(p, M, cols, d);
  a.part = parts.part;
  return launch<kPartial>(a, p, StreamSum{}, std::min(a.items, d.sms), stream);
}

bool i8_cluster_suits(const StreamSum& s, int K, const LoraDevice& d) {
  // U's columns start on the 16-byte grid
  return (!s.gate || s.N % 16 == 0) && cluster_pays(cluster_tiles(s, K, kBlockRows, false, d), d.sms);
}

int i8_cluster(const NarrowStream& p, const StreamSum& s, const LoraDevice& d,
               cudaStream_t stream) {
  Args a{};
  static_cast<Tiles&>(a) = cluster_tiles(s, p.K, kBlockRows, false, d);
  if (a.chunks == 0) return GEMM_ERR_ARG;
  lay_out(a, (a.kb + a.chunks - 1) / a.chunks, true);
  return s.gate ? launch<kScaledGate>(a, p, s, a.items, stream)
                : launch<kScaled>(a, p, s, a.items, stream);
}

}  // namespace gb300
