// narrow_stream.cu -- products with few rows or few tiles, of halves or of 8-bit
// integers: W is the M operand of tcgen05.mma (128 of its columns), the rows of X the N
// operand, K is cut into chunks that go to different SMs.
//
// Two ways to add the chunks up:
//   cluster    as many chunks as a cluster has CTAs (1, 2, 4 or 8), each CTA one chunk of
//              one tile; the sums meet in shared memory, each CTA adds up its share of the
//              outputs through distributed shared memory, finishes and stores them.  One
//              launch, no partial sums in global memory: for products that one wave
//              of CTAs covers
//   partial    (8-bit integers; of halves lora_stream.cu) fp32 partial sums of any number
//              of chunks over persistent CTAs, added up by stream_sum.cu: for W that
//              takes longer than that, where evenly shared work counts for more
// A gate's unit is 64 of its columns and the 64 that they gate, so that a CTA of the cluster
// form has both sums of an output.
//
// 8-bit integers.  This card's tensor cores run them far below halves, and every 8-bit
// integer is a half exactly: W and X come from HBM as bytes by TMA and become halves on
// their way through shared memory.  Products are exact, and so are the fp32 sums while
// they stay below 2^24 (always for K <= 1024).  Two groups of eight warps convert 64 k of
// each step, into two operand buffers of their own, so that the waits and the proxy
// fence of one pass beside the other's work.
//
// Steps are 128 deep, and a step's tile of W (and of X) is one TMA instruction where
// the sizes allow (maps of three dimensions): the thread that issues them takes about
// 0.1 us for each, so that with 64-deep steps of three instructions a CTA took in 16 KB of
// W in 0.31 us, whatever the bytes.  The first loads are issued before tensor memory is
// allocated and the CTA's threads have met.
//
// Shared memory.  Halves: ring stages of W, two 64-column blocks [128 k][64 halves]
// (MN-major, 128-byte swizzle, LBO 16 KB), or of a W stored transposed two 64-deep blocks
// [128 columns][64 halves] (K-major); then X, two 64-deep blocks [row][64 halves]
// (K-major), or 64-row blocks [128 k][64 halves].  Integers: four operand buffers of
// 64 k (W as two blocks [64 k][64 halves], X as [row][64 halves]), then the ring of
// raw steps, W as [128 k][128 bytes] (of a gate, in the cluster form, two blocks [128 k][64
// bytes]) and X as [row][128 bytes], swizzled over their rows.  Each group converts
// its half of every step.
#include "i8_convert.cuh"
#include "stream_finish.cuh"

namespace gb300 {
namespace {

constexpr int kStepK = 128;
constexpr int kHalfW = kStepK * 256;        // 128 columns of a step as halves
constexpr int kByteW = kStepK * 128;        // as bytes
constexpr int kOpW = kHalfW / 2;            // of an operand buffer
constexpr int kMaxStages = 8;
constexpr int kGroups = 2;                  // of converting warps
constexpr int kGroupWarps = 8;
constexpr int kBufs = 2 * kGroups;          // operand buffers
constexpr int kSmemMax = 232448;
constexpr int kPartial = -1;
// how an output is finished (cluster form)
enum Finish { kHalf, kFloat, kGate, kGateGrad, kScaled, kScaledGate };

struct Args {
  int M, N;                     // rows; columns of W that exist
  int kb, chunks, units, items; // steps, chunks, units, blocks x units x chunks
  int stages, raw_bytes, x_bytes, op_bytes, n_cols, acc_cols;
  int unit_cols;                // first columns of units apart
  int rows;                     // rows of a block (at most)
  int bar_off;
  bool trans_w, trans_x, reread;
  bool one_w, one_x;            // the step's tile is one instruction
  bool vec;
  float* part;
  unsigned long long wait_limit_ns;
  DeviceStatus* status;
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}

template <bool I8>
constexpr int threads() {
  return 64 + 32 * (I8 ? kGroupWarps * kGroups : 8);
}

template <bool I8, int FIN>
__global__ void __launch_bounds__(threads<I8>(), 1)
    narrow_stream_kernel(const __grid_constant__ CUtensorMap tmW,
                         const __grid_constant__ CUtensorMap tmX, const Args p, const StreamSum fin) {
  constexpr int kEpi = I8 ? kGroupWarps * kGroups : 8;   // warps that write sums (and convert)
  constexpr int kRawW = I8 ? kByteW : kHalfW;
  constexpr bool kWide = I8 && FIN != kScaledGate;   // raw rows of W are 128 bytes wide
  constexpr bool kCluster = FIN != kPartial;
  constexpr bool kPaired = FIN == kGate || FIN == kGateGrad || FIN == kScaledGate;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw0 = smem_addr(smem_raw);
  const uint32_t base = (raw0 + 1023u) & ~1023u;
  uint8_t* const base_ptr = smem_raw + (base - raw0);
  const int S = p.stages;
  const int warp = warp_id_uniform(), lane = static_cast<int>(lane_id());
  const uint32_t raws = base + static_cast<uint32_t>(I8 ? kBufs * p.op_bytes : 0);
  const uint32_t bars = base + static_cast<uint32_t>(p.bar_off);
  auto full_bar = [&](int s) { return bars + 8u * s; };
  auto empty_bar = [&](int s) { return bars + 8u * (kMaxStages + s); };
  auto op_full = [&](int b) { return bars + 8u * (2 * kMaxStages + b); };
  auto op_empty = [&](int b) { return bars + 8u * (2 * kMaxStages + kBufs + b); };
  const uint32_t acc_full = bars + 8u * (2 * kMaxStages + 2 * kBufs);
  const uint32_t acc_empty = acc_full + 8u, done_bar = acc_full + 16u;
  uint8_t* const tmem_ptr = base_ptr + p.bar_off + 8 * (2 * kMaxStages + 2 * kBufs + 3);
  const unsigned long long limit = p.wait_limit_ns;
  DeviceStatus* const st = p.status;
  auto first_step = [&](int it) { return it % p.chunks * p.kb / p.chunks; };
  auto end_step = [&](int it) { return (it % p.chunks + 1) * p.kb / p.chunks; };
  // one step's loads into stage s
  const uint64_t policy = l2_evict_first_policy();
  auto load_step = [&](int s, int n0, int row0, int step) {
    const uint32_t dst = raws + static_cast<uint32_t>(s * p.raw_bytes), bar = full_bar(s);
    const int k = step * kStepK;
    mbar_arrive_expect_tx(bar, static_cast<uint32_t>(p.raw_bytes));
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
    if (I8) {
      if (kWide)
        w2(dst, n0, k);
      else
        w3(n0, k, 0);              // [gate or up][k][column]
    } else if (p.trans_w) {
      if (p.one_w) {
        w3(0, n0, 2 * step);       // [64 k][column][k]
      } else {
        w2(dst, k, n0);
        w2(dst + kRawW / 2, k + 64, n0);
      }
    } else if (p.one_w) {
      if (kPaired)
        w3(n0, k, 0);              // [gate or up][k][column]
      else
        w3(0, k, n0 / 64);         // [64 columns][k][column]
    } else {
      w2(dst, n0, k);
      w2(dst + kRawW / 2, n0 + 64, k);
    }
    const uint32_t x = dst + kRawW;
    if (I8) {
      tma_load_2d(x, &tmX, bar, k, row0);
    } else if (p.trans_x) {
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
  auto item_n0 = [&](int it) { return it / p.chunks % p.units * p.unit_cols; };
  auto item_row0 = [&](int it) { return it / p.chunks / p.units * p.rows; };
  if (warp == 0) {
    // barriers, a lane each
    if (lane < S) {
      mbar_init(full_bar(lane), 1u);
      // the converting warps, or an MMA commit
      mbar_init(empty_bar(lane), I8 ? kGroups * kGroupWarps : 1u);
    }
    if (I8 && lane < kBufs) {
      mbar_init(op_full(lane), kGroupWarps);
      mbar_init(op_empty(lane), 1u);
    }
    if (lane == 31) {
      mbar_init(acc_full, 1u);
      mbar_init(acc_empty, static_cast<uint32_t>(kEpi));
      mbar_init(done_bar, 1u);
    }
    fence_barrier_init();
    fence_proxy_async_smem();
    __syncwarp();
    griddep_wait();   // copies onto the 16-byte grid, if any
    // the first item's first steps: their stages are empty
    if (lane == 0) {
      const int it = blockIdx.x, n = min(S, end_step(it) - first_step(it));
      for (int s = 0; s < n; ++s) load_step(s, item_n0(it), item_row0(it), first_step(it) + s);
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
  if (warp > 0) griddep_wait();   // (what the results are joined with)
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_ptr);

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      // (the first item's first steps are on their way)
      int skip = min(S, end_step(blockIdx.x) - first_step(blockIdx.x)), s = 0;
      uint32_t phase = 0, issued = 0;
      bool ok = true;
      for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
        const int n0 = item_n0(it), row0 = item_row0(it), end = end_step(it);
        for (int step = first_step(it); step < end; ++step) {
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
      constexpr uint32_t kMmas = I8 ? 4 : 8;      // of 16 k
      const int ring = I8 ? kBufs : S, halves = I8 ? 2 : 1;   // (operand buffers are half steps)
      const uint32_t ring0 = I8 ? base : raws;
      const uint32_t stride = static_cast<uint32_t>(I8 ? p.op_bytes : p.raw_bytes) >> 4;
      const uint32_t first_bar = I8 ? op_full(0) : full_bar(0);
      const uint32_t free_bar = I8 ? op_empty(0) : empty_bar(0);
      const bool tw = !I8 && p.trans_w, tx = !I8 && p.trans_x;
      const uint32_t x0 = ring0 + (I8 ? kOpW : kHalfW);
      const uint64_t wd0 = smem_desc_sw128(ring0, tw ? 16u : (I8 ? 8192u : 16384u), 1024u);
      const uint64_t xd0 = smem_desc_sw128(x0, tx ? 16384u : 16u, 1024u);
      // 16 k and 64 k on, in 16 bytes
      const uint32_t wk = tw ? 2u : 128u, wq = tw ? 1024u : 512u;
      const uint32_t xk = tx ? 128u : 2u, xq = tx ? 512u : static_cast<uint32_t>(p.n_cols) * 8u;
      int s = 0;
      uint32_t phase = 0, local = 0, off = 0;
      bool ok = true, ready = false;
      for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x, ++local) {
        int left = (end_step(it) - first_step(it)) * halves;
        if (!wait_parity(acc_empty, (local & 1u) ^ 1u, limit, st, 72)) break;
        tc_fence_after();
        for (uint32_t acc = 0; left > 0; --left) {
          if (!ready && !wait_parity(first_bar + 8u * s, phase, limit, st, 73)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t done = free_bar + 8u * s;
          const uint64_t wd = wd0 + off, xd = xd0 + off;
          off += stride;
          if (++s == ring) {
            s = 0;
            off = 0;
            phase ^= 1u;
          }
          ready = mbar_try_wait(first_bar + 8u * s, phase);
#pragma unroll
          for (uint32_t kk = 0; kk < kMmas; ++kk) {
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
    // ------------------------------------------------------------ converters, sums
    const int ew = warp - 2, t = static_cast<int>(threadIdx.x) - 64;
    const int quad = warp & 3, part = ew >> 2;
    uint32_t step = 0, local = 0;
    bool ok = true;
    for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x, ++local) {
      if constexpr (I8) {
        const int group = ew / kGroupWarps, tg = t % (32 * kGroupWarps);
        const uint32_t end = step + static_cast<uint32_t>(end_step(it) - first_step(it));
        for (; step < end; ++step) {   // (steps are counted over all items)
          const int s = static_cast<int>(step % S);
          const uint32_t n = 2 * step + group;
          const int b = static_cast<int>(n % kBufs);
          if (!wait_parity(full_bar(s), (step / S) & 1u, limit, st, 75) ||
              !wait_parity(op_empty(b), ((n / kBufs) & 1u) ^ 1u, limit, st, 76)) {
            ok = false;
            break;
          }
          const uint8_t* const src =
              base_ptr + (raws - base) + static_cast<size_t>(s) * p.raw_bytes;
          uint8_t* const op = base_ptr + static_cast<size_t>(b) * p.op_bytes;
          // X, 16 bytes each: four to a row; the eight threads of two rows store to eight
          // bank groups, pieces being swizzled by the row
          const int r4 = tg >> 2, j = (tg & 3) * 2;
          const int at0 = r4 * 128 + ((j ^ (r4 & 7)) << 4);
          const int at1 = r4 * 128 + (((j + 1) ^ (r4 & 7)) << 4);
          // this group's 64 k: rows of W, the first or second half of X's
          const int raw_x = r4 * 128 + ((((tg & 3) + 4 * group) ^ (r4 & 7)) << 4);
          const int raw_w = kWide ? group * 8192 + (tg >> 3) * 128 + (((tg & 7) ^ ((tg >> 3) & 7)) << 4)
                                  : group * 4096 + r4 * 64 + (((tg & 3) ^ ((r4 >> 1) & 3)) << 4);
          uint4 v[2];
#pragma unroll
          for (int i = 0; i < 2; ++i)
            v[i] = *reinterpret_cast<const uint4*>(src + raw_w + i * (kWide ? 4096 : 8192));
          if constexpr (kWide) {
            // W: eight to a row of k, four for either block; those of the second store
            // their two pieces the other way round, again for the banks' sake
            const int k8 = tg >> 3;
            const bool second = (tg & 4) != 0;
            const int w0 = (second ? 8192 : 0) + k8 * 128 + ((j ^ (k8 & 7)) << 4);
            const int w1 = (second ? 8192 : 0) + k8 * 128 + (((j + 1) ^ (k8 & 7)) << 4);
#pragma unroll
            for (int i = 0; i < 2; ++i) {   // 32 rows of k each
              uint4 a, c;
              i8_halves16(v[i], a, c);
              *reinterpret_cast<uint4*>(op + i * 4096 + (second ? w1 : w0)) = second ? c : a;
              *reinterpret_cast<uint4*>(op + i * 4096 + (second ? w0 : w1)) = second ? a : c;
            }
          } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {   // a block each
              uint4 a, c;
              i8_halves16(v[i], a, c);
              *reinterpret_cast<uint4*>(op + i * 8192 + at0) = a;
              *reinterpret_cast<uint4*>(op + i * 8192 + at1) = c;
            }
          }
          for (int r = 0; r + r4 < p.n_cols; r += 8 * kGroupWarps) {
            uint4 a, c;
            i8_halves16(*reinterpret_cast<const uint4*>(src + kRawW + raw_x + r * 128), a, c);
            *reinterpret_cast<uint4*>(op + kOpW + r * 128 + at0) = a;
            *reinterpret_cast<uint4*>(op + kOpW + r * 128 + at1) = c;
          }
          fence_proxy_async_smem();   // generic writes -> tensor-core reads
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(empty_bar(s));
            mbar_arrive(op_full(b));
          }
        }
      }
      if (!ok || !wait_parity(acc_full, local & 1u, limit, st, 77)) {
        ok = false;
        break;
      }
      tc_fence_after();
      // sums of 32 columns of W (lanes) by rows of X, to global memory or, the ring
      // being done with, to the start of shared memory: [row][128]
      const uint32_t d0 = tmem + (static_cast<uint32_t>(32 * quad) << 16);
      float* const out =
          kCluster ? reinterpret_cast<float*>(base_ptr) + 32 * quad + lane
                   : p.part + static_cast<long long>(it) * p.rows * 128 + 32 * quad + lane;
      const int rows = min(p.rows, p.M - it / p.chunks / p.units * p.rows);
      for (int r0 = 16 * part; r0 < rows; r0 += 4 * kEpi) {   // n_cols is a multiple of 16
        uint32_t g[8], h[8];
        tmem_ld_32x32b_x8(d0 + r0, g);
        tmem_ld_32x32b_x8(d0 + r0 + 8, h);
        tmem_wait_ld2(g, h);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (r0 + i < rows) out[(r0 + i) * 128] = __uint_as_float(g[i]);
          if (r0 + 8 + i < rows) out[(r0 + 8 + i) * 128] = __uint_as_float(h[i]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty);
    }
  }
  if constexpr (kCluster) {
    __syncwarp();
    cluster_sync();   // every chunk's sums are in its CTA's shared memory
    constexpr int kGateOf = FIN == kGateGrad ? 2 : (kPaired ? 1 : 0);
    constexpr int kQuads = kPaired ? 16 : 32;   // quads of output columns in a unit
    const int it = blockIdx.x, rank = it % p.chunks;
    const int unit = it / p.chunks % p.units, row0 = it / p.chunks / p.units * p.rows;
    const int total = min(p.rows, p.M - row0) * kQuads;
    for (int i = rank * total / p.chunks + static_cast<int>(threadIdx.x);
         i < (rank + 1) * total / p.chunks; i += threads<I8>()) {
      const int r = i / kQuads, q = i % kQuads;
      const int c = unit * p.unit_cols + 4 * q, n = min(4, fin.N - c);
      if (n <= 0) continue;
      const uint32_t at = base + static_cast<uint32_t>((r * 128 + 4 * q) * 4);
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
          if (kPaired) add(u, ld_cluster_f4(peer + 256));
        }
      stream_finish<kGateOf, FIN == kFloat, FIN == kScaled || FIN == kScaledGate, 4>(
          fin, row0 + r, c, n, p.vec && n == 4, s, u);
    }
    cluster_sync();   // nobody leaves while its sums are being read
  } else {
    __syncthreads();
  }
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, p.acc_cols);
}

// ------------------------------------------------------------------- plans
constexpr int kHalfRows = 256, kI8Rows = 128;   // rows of a block

// Stages, buffers and the place of the barriers, for `steps` steps a CTA at most.
void lay_out(Args& a, bool i8, int steps, bool cluster) {
  a.n_cols = ((a.rows < a.M ? a.rows : a.M) + 15) / 16 * 16;
  a.acc_cols = 32;
  while (a.acc_cols < a.n_cols) a.acc_cols *= 2;
  a.x_bytes = i8          ? a.n_cols * 128
              : a.trans_x ? (a.n_cols + 63) / 64 * 16384
                          : a.n_cols * 256;
  a.raw_bytes = (i8 ? kByteW : kHalfW) + a.x_bytes;
  a.op_bytes = i8 ? kOpW + a.n_cols * 128 : 0;
  a.stages = std::min({kMaxStages, (kSmemMax - 2048 - kBufs * a.op_bytes) / a.raw_bytes, steps});
  int bytes = kBufs * a.op_bytes + a.stages * a.raw_bytes;
  if (cluster) bytes = std::max(bytes, a.n_cols * 512);
  a.bar_off = bytes;
}

// The cluster form's chunks for `tiles` tiles of `steps` steps: as many as one wave of
// CTAs leaves room for (76, 36 and 15 clusters of 2, 4 and 8 CTAs fit on 152 SMs); 0: it
// does not suit.
int cluster_chunks(long long tiles, int steps, int sms) {
  if (tiles > sms) return 0;
  int best = 1;
  for (int c = 2; c <= 8; c *= 2)
    if (tiles * c <= (c <= 2 ? sms : c == 4 ? sms - 8 : sms - 32) && steps >= c) best = c;
  return best;
}

template <bool I8, int FIN>
int launch(const Args& a, const StreamSum& fin, const CUtensorMap& tmW, const CUtensorMap& tmX,
           int grid, bool early, cudaStream_t stream) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return GEMM_ERR_CUDA;
  static bool configured[64] = {};
  if (dev < 64 && !configured[dev]) {
    if (cudaFuncSetAttribute(narrow_stream_kernel<I8, FIN>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax) != cudaSuccess)
      return GEMM_ERR_CUDA;
    configured[dev] = true;
  }
  cudaLaunchAttribute attr[2];
  unsigned int n = 0;
  if (FIN != kPartial) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = static_cast<unsigned>(a.chunks);
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (early) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(threads<I8>(), 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(a.bar_off) + 2048;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return counted_launch(cudaLaunchKernelEx(&cfg, narrow_stream_kernel<I8, FIN>, tmW, tmX, a, fin)) ==
                 cudaSuccess
             ? GEMM_OK
             : GEMM_ERR_CUDA;
}

// The maps of the operands.  Three dimensions, so that a step is one instruction,
// where they stay inside the matrix: 64-column (or 64-row, 64-deep) blocks as the third
// dimension of one whose size is a multiple of 64; a gate's columns and those it
// gates.  `paired`: the latter, U's columns `up` after G's.
int make_maps(Args& a, bool i8, const void* W, long long ldw, const void* X, long long ldx, int K,
              bool paired, int up, CUtensorMap* tmW, CUtensorMap* tmX) {
  if (i8) {
    if (int rc = paired ? encode_map_3d(tmW, 1, W, {up, K, 2}, {ldw, up}, {64, kStepK, 2})
                        : encode_map_3d(tmW, 1, W, {a.N, K, 0}, {ldw, 0}, {128, kStepK, 0}))
      return rc;
    return encode_map_3d(tmX, 1, X, {K, a.M, 0}, {ldx, 0}, {kStepK, a.n_cols, 0});
  }
  int rc;
  if (a.trans_w) {
    a.one_w = K % 64 == 0;
    rc = a.one_w ? encode_map_3d(tmW, 2, W, {64, a.N, K / 64}, {ldw, 64}, {64, 128, 2})
                 : encode_map_3d(tmW, 2, W, {K, a.N, 0}, {ldw, 0}, {64, 128, 0});
  } else if (paired) {
    a.one_w = true;
    rc = encode_map_3d(tmW, 2, W, {up, K, 2}, {ldw, up}, {64, kStepK, 2});
  } else {
    a.one_w = a.N % 64 == 0;
    rc = a.one_w ? encode_map_3d(tmW, 2, W, {64, K, a.N / 64}, {ldw, 64}, {64, kStepK, 2})
                 : encode_map_3d(tmW, 2, W, {a.N, K, 0}, {ldw, 0}, {64, kStepK, 0});
  }
  if (rc) return rc;
  if (a.trans_x) {
    a.one_x = a.M % 64 == 0;
    return a.one_x ? encode_map_3d(tmX, 2, X, {64, K, a.M / 64}, {ldx, 64},
                                   {64, kStepK, (a.n_cols + 63) / 64})
                   : encode_map_3d(tmX, 2, X, {a.M, K, 0}, {ldx, 0}, {64, kStepK, 0});
  }
  a.one_x = K % 64 == 0;
  return a.one_x ? encode_map_3d(tmX, 2, X, {64, a.M, K / 64}, {ldx, 64}, {64, a.n_cols, 2})
                 : encode_map_3d(tmX, 2, X, {K, a.M, 0}, {ldx, 0}, {64, a.n_cols, 0});
}

int block_rows(bool i8) { return i8 ? kI8Rows : kHalfRows; }

Args plan_partial(const NarrowStream& p, int M, int cols, bool fold, int sms) {
  Args a{};
  const int rows = block_rows(p.i8), blocks = (M + rows - 1) / rows;
  a.M = M;
  a.N = cols;
  a.rows = std::min(M, rows);
  a.kb = (p.K + kStepK - 1) / kStepK;
  a.units = (cols + 127) / 128;
  a.unit_cols = 128;
  a.trans_w = p.trans_w;
  a.trans_x = p.trans_x;
  // (in 64-deep k-blocks of halves, 16 KB of W)
  a.chunks = std::min(a.kb, plan_chunks(a.units, blocks, p.i8 ? a.kb : 2 * a.kb, a.rows, sms,
                                        fold ? (p.K + kFoldDepth - 1) / kFoldDepth : 1));
  a.items = blocks * a.units * a.chunks;
  a.reread = blocks > 1;
  lay_out(a, p.i8, kMaxStages, false);
  return a;
}

}  // namespace

StreamParts narrow_parts(const NarrowStream& p, int M, int cols, bool fold, int sms) {
  const Args a = plan_partial(p, M, cols, fold, sms);
  return StreamParts{nullptr, a.chunks, a.units, a.rows,
                     4 * static_cast<size_t>(a.items) * a.rows * 128, block_rows(p.i8)};
}

int narrow_partial(const NarrowStream& p, int M, int cols, bool fold, const StreamParts& parts,
                   const LoraDevice& d, bool early, cudaStream_t stream) {
  Args a = plan_partial(p, M, cols, fold, d.sms);
  a.part = parts.part;
  a.wait_limit_ns = d.wait_limit_ns;
  a.status = d.status;
  CUtensorMap tmW{}, tmX{};
  if (int rc = make_maps(a, p.i8, p.W, p.ldw, p.X, p.ldx, p.K, false, 0, &tmW, &tmX)) return rc;
  const int grid = std::min(a.items, d.sms);
  return p.i8 ? launch<true, kPartial>(a, StreamSum{}, tmW, tmX, grid, early, stream)
              : launch<false, kPartial>(a, StreamSum{}, tmW, tmX, grid, early, stream);
}

bool narrow_cluster_suits(bool i8, int M, int N, int K, int gate, bool f32, int sms) {
  // U's columns start on TMA's 16-byte grid
  if (gate && N % (i8 ? 16 : 8) != 0) return false;
  const int rows = block_rows(i8), unit = gate ? 64 : 128;
  const long long tiles = static_cast<long long>((M + rows - 1) / rows) * ((N + unit - 1) / unit);
  const int chunks = cluster_chunks(tiles, (K + kStepK - 1) / kStepK, sms);
  return chunks > 0 && (!f32 || (K + chunks - 1) / chunks + kStepK <= kFoldDepth);
}

int narrow_cluster(const NarrowStream& p, const StreamSum& s, const LoraDevice& d, bool early,
                   cudaStream_t stream) {
  const int rows = block_rows(p.i8), blocks = (s.M + rows - 1) / rows;
  Args a{};
  a.M = s.M;
  a.N = s.gate ? 2 * s.N : s.N;
  a.rows = std::min(s.M, rows);
  a.kb = (p.K + kStepK - 1) / kStepK;
  a.unit_cols = s.gate ? 64 : 128;
  a.units = (s.N + a.unit_cols - 1) / a.unit_cols;
  a.trans_w = p.trans_w;
  a.trans_x = p.trans_x;
  a.chunks = cluster_chunks(1ll * blocks * a.units, a.kb, d.sms);
  if (a.chunks == 0) return GEMM_ERR_ARG;
  a.items = blocks * a.units * a.chunks;
  a.reread = blocks > 1;
  lay_out(a, p.i8, (a.kb + a.chunks - 1) / a.chunks, true);
  uintptr_t bits = reinterpret_cast<uintptr_t>(s.C);
  a.vec = s.ldc % 4 == 0;
  if (s.gate == 2) {
    bits |= reinterpret_cast<uintptr_t>(s.g.dC) | reinterpret_cast<uintptr_t>(s.g.dU);
    a.vec = a.vec && s.g.lddc % 4 == 0;
  }
  a.vec = a.vec && bits % (s.f32 ? 16 : 8) == 0;
  a.wait_limit_ns = d.wait_limit_ns;
  a.status = d.status;
  CUtensorMap tmW{}, tmX{};
  if (int rc = make_maps(a, p.i8, p.W, p.ldw, p.X, p.ldx, p.K, s.gate != 0, s.N, &tmW, &tmX))
    return rc;
  if (p.i8)
    return s.gate ? launch<true, kScaledGate>(a, s, tmW, tmX, a.items, early, stream)
                  : launch<true, kScaled>(a, s, tmW, tmX, a.items, early, stream);
  return s.gate == 2 ? launch<false, kGateGrad>(a, s, tmW, tmX, a.items, early, stream)
         : s.gate    ? launch<false, kGate>(a, s, tmW, tmX, a.items, early, stream)
         : s.f32     ? launch<false, kFloat>(a, s, tmW, tmX, a.items, early, stream)
                     : launch<false, kHalf>(a, s, tmW, tmX, a.items, early, stream);
}

}  // namespace gb300
