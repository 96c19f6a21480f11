// i8_stream.cu -- products in 8-bit integers with few rows or few tiles: fp32
// partial sums by (128 rows, 128 columns, K chunk), added up by stream_sum.cu.
//
// This card's tensor cores run 8-bit integers far below halves, and every 8-bit integer
// is a half exactly: W and X come from HBM as bytes by TMA and become halves on their way
// through shared memory, where tcgen05.mma reads them (W as the M operand, the rows of
// X as the N operand).  Products are exact, and so are the fp32 sums while they stay
// below 2^24 (always for K <= 1024).
//
//   byte b = q + 128 (q xor 0x80)  ->  half 0x6400 | b = 1024 + b  ->  minus 1152 = q
// two byte permutes and two packed subtractions for four integers.
//
// Warps: a TMA producer, an MMA issuer, and eight that convert a 128-deep step (16 KB
// of W) from the ring of raw steps into one of two buffers of operands, and at an
// item's end write its sums.  A conversion is 30 instructions per 16 bytes: 0.15 us a
// step on an SM's four schedulers, while HBM brings one in 0.37 us.
//
// Shared memory: raw steps of W [128 k][128 bytes] and X [row][128 bytes], as they lie
// in memory; operand buffers as in lora_stream.cu, for each 64-deep half two 64-column
// blocks of W (MN-major, 128-byte swizzle, LBO 8 KB) and 64 halves of k of each row of X
// (K-major).
#include <cuda_fp16.h>

#include "stream.h"

namespace gb300 {
namespace {

constexpr int kRows = 128;                  // rows of a block (N of the MMA)
constexpr int kStepK = 128;
constexpr int kRawW = kStepK * 128;         // 16 KB
constexpr int kOpW = 2 * kRawW;             // 32 KB
constexpr int kMaxStages = 10;
constexpr int kConv = 8;
constexpr int kThreads = 32 * (2 + kConv);
constexpr int kSmemMax = 232448;

struct Args {
  int M, N;
  int kb, chunks, units, items;
  int stages, raw_bytes, op_bytes, n_cols;
  int block_rows;
  float* part;
  unsigned long long wait_limit_ns;
  DeviceStatus* status;
};

// Four 8-bit integers as halves.
__device__ __forceinline__ uint2 halves_of(uint32_t w) {
  const uint32_t b = w ^ 0x80808080u;
  const uint32_t lo = __byte_perm(b, 0x64646464u, 0x4140), hi = __byte_perm(b, 0x64646464u, 0x4342);
  const __half2 off = __half2half2(__ushort_as_half(0x6480));
  __half2 l, h;
  memcpy(&l, &lo, 4);
  memcpy(&h, &hi, 4);
  l = __hsub2(l, off);
  h = __hsub2(h, off);
  uint2 r;
  memcpy(&r.x, &l, 4);
  memcpy(&r.y, &h, 4);
  return r;
}

// 16 integers (chunk c of a 128-byte row) to halves 16 c .. of the operand row `row`:
// two 16-byte pieces of one of its four 128-byte rows (`row_of(block)`, block = 64 halves).
// Threads of the second 64 halves store their pieces in the other order, so that the
// eight threads of a row touch all banks.
__device__ __forceinline__ void convert16(uint4 raw, uint8_t* dst_row, int c, int row) {
  const uint2 a = halves_of(raw.x), b = halves_of(raw.y), d = halves_of(raw.z), e = halves_of(raw.w);
  const uint4 first = make_uint4(a.x, a.y, b.x, b.y), second = make_uint4(d.x, d.y, e.x, e.y);
  const int j = (c & 3) * 2;
  uint8_t* const p0 = dst_row + ((j ^ (row & 7)) << 4);
  uint8_t* const p1 = dst_row + (((j + 1) ^ (row & 7)) << 4);
  const bool swap = c >= 4;
  *reinterpret_cast<uint4*>(swap ? p1 : p0) = swap ? second : first;
  *reinterpret_cast<uint4*>(swap ? p0 : p1) = swap ? first : second;
}

__global__ void __launch_bounds__(kThreads, 1)
    i8_stream_kernel(const __grid_constant__ CUtensorMap tmW,
                     const __grid_constant__ CUtensorMap tmX, const Args p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw0 = smem_addr(smem_raw);
  const uint32_t base = (raw0 + 1023u) & ~1023u;
  uint8_t* const base_ptr = smem_raw + (base - raw0);
  const int S = p.stages;
  const int warp = warp_id_uniform(), lane = static_cast<int>(lane_id());
  // operand buffers first (1024-byte aligned), then the raw steps, then the barriers
  const uint32_t raws = base + 2u * p.op_bytes;
  const uint32_t bars = raws + static_cast<uint32_t>(S * p.raw_bytes);
  auto raw_full = [&](int s) { return bars + 8u * s; };
  auto raw_empty = [&](int s) { return bars + 8u * (kMaxStages + s); };
  auto op_full = [&](uint32_t b) { return bars + 8u * (2 * kMaxStages + b); };
  auto op_empty = [&](uint32_t b) { return bars + 8u * (2 * kMaxStages + 2 + b); };
  const uint32_t acc_full = bars + 8u * (2 * kMaxStages + 4);
  const uint32_t acc_empty = bars + 8u * (2 * kMaxStages + 5);
  const uint32_t done_bar = bars + 8u * (2 * kMaxStages + 6);
  uint8_t* const tmem_ptr = base_ptr + (bars - base) + 8 * (2 * kMaxStages + 7);
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(raw_full(s), 1u);
      mbar_init(raw_empty(s), static_cast<uint32_t>(kConv));
    }
    for (uint32_t b = 0; b < 2; ++b) {
      mbar_init(op_full(b), static_cast<uint32_t>(kConv));
      mbar_init(op_empty(b), 1u);
    }
    mbar_init(acc_full, 1u);
    mbar_init(acc_empty, static_cast<uint32_t>(kConv));
    mbar_init(done_bar, 1u);
    fence_barrier_init();
    fence_proxy_async_smem();
    prefetch_tensormap(&tmW);
    prefetch_tensormap(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(tmem_ptr), 128);
    tmem_relinquish();
    griddep_launch_dependents();   // only now: see lora_stream.cu
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_wait();   // copies onto the 16-byte grid, if any
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_ptr);
  const unsigned long long limit = p.wait_limit_ns;
  DeviceStatus* const st = p.status;

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t policy = l2_evict_first_policy();
      int s = 0;
      uint32_t phase = 0, issued = 0;
      bool ok = true;
      for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
        const int c = it % p.chunks, n0 = it / p.chunks % p.units * 128;
        const int row0 = it / p.chunks / p.units * kRows;
        for (int kb = c * p.kb / p.chunks; kb < (c + 1) * p.kb / p.chunks; ++kb) {
          if (!wait_parity(raw_empty(s), phase ^ 1u, limit, st, 70)) {
            ok = false;
            break;
          }
          const uint32_t dst = raws + static_cast<uint32_t>(s * p.raw_bytes);
          mbar_arrive_expect_tx(raw_full(s), static_cast<uint32_t>(p.raw_bytes));
          // W evict-first when no other block of rows reads it
          if (p.M <= kRows)
            tma_load_2d_hint(dst, &tmW, raw_full(s), n0, kb * kStepK, policy);
          else
            tma_load_2d(dst, &tmW, raw_full(s), n0, kb * kStepK);
          tma_load_2d(dst + kRawW, &tmX, raw_full(s), kb * kStepK, row0);
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
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = make_idesc(0u, 128u, static_cast<uint32_t>(p.n_cols), 1u, 0u);
      uint32_t step = 0, local = 0;
      bool ok = true;
      for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x, ++local) {
        const int c = it % p.chunks;
        const int kb0 = c * p.kb / p.chunks, kb1 = (c + 1) * p.kb / p.chunks;
        if (!wait_parity(acc_empty, (local & 1u) ^ 1u, limit, st, 72)) break;
        tc_fence_after();
        for (int kb = kb0; kb < kb1; ++kb, ++step) {
          const uint32_t b = step & 1u;
          if (!wait_parity(op_full(b), (step >> 1) & 1u, limit, st, 73)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t w0 = base + b * p.op_bytes, x0 = w0 + kOpW;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_f16_ss(tmem, smem_desc_sw128(w0 + (kk >> 2) * kRawW + (kk & 3) * 2048, 8192u, 1024u),
                       smem_desc_sw128(x0 + (kk >> 2) * p.n_cols * 128 + (kk & 3) * 32, 16u, 1024u),
                       idesc, (kb > kb0 || kk > 0) ? 1u : 0u);
          mma_commit(op_empty(b));
        }
        if (!ok) break;
        mma_commit(acc_full);
      }
      mma_commit(done_bar);
      settle_wait(done_bar, 0u, st, 74);
    }
    __syncwarp();
  } else {
    const int t = static_cast<int>(threadIdx.x) - 64;   // 0 .. 255
    const int quad = warp & 3, part = (warp - 2) >> 2;
    int s = 0;
    uint32_t phase = 0, step = 0, local = 0;
    bool ok = true;
    for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x, ++local) {
      const int c0 = it % p.chunks;
      for (int kb = c0 * p.kb / p.chunks; kb < (c0 + 1) * p.kb / p.chunks; ++kb, ++step) {
        const uint32_t b = step & 1u;
        if (!wait_parity(raw_full(s), phase, limit, st, 75) ||
            !wait_parity(op_empty(b), ((step >> 1) & 1u) ^ 1u, limit, st, 76)) {
          ok = false;
          break;
        }
        const uint8_t* const src = base_ptr + (raws - base) + static_cast<size_t>(s) * p.raw_bytes;
        uint8_t* const op = base_ptr + static_cast<size_t>(b) * p.op_bytes;
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const uint4*>(src + (t + 256 * i) * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int k = (t >> 3) + 32 * i, c = t & 7;
          // [64-deep half][64-column block][k % 64][128 bytes]
          convert16(v[i], op + ((k >> 6) * 2 + (c >> 2)) * 8192 + (k & 63) * 128, c, k);
        }
        for (int id = t; id < 8 * p.n_cols; id += 256) {
          const int r = id >> 3, c = id & 7;
          const uint4 x = *reinterpret_cast<const uint4*>(src + kRawW + id * 16);
          convert16(x, op + kOpW + ((c >> 2) * p.n_cols + r) * 128, c, r);
        }
        fence_proxy_async_smem();   // generic writes -> tensor-core reads
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(raw_empty(s));
          mbar_arrive(op_full(b));
        }
        if (++s == S) {
          s = 0;
          phase ^= 1u;
        }
      }
      if (!ok || !wait_parity(acc_full, local & 1u, limit, st, 77)) break;
      tc_fence_after();
      const uint32_t d0 = tmem + (static_cast<uint32_t>(32 * quad) << 16);
      float* const out =
          p.part + static_cast<long long>(it) * p.block_rows * 128 + 32 * quad + lane;
      const int rows = min(kRows, p.M - it / p.chunks / p.units * kRows);
      for (int r0 = 16 * part; r0 < rows; r0 += 32) {   // n_cols is a multiple of 16
        uint32_t g[8], h[8];
        tmem_ld_32x32b_x8(d0 + r0, g);
        tmem_ld_32x32b_x8(d0 + r0 + 8, h);
        tmem_wait_ld2(g, h);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (r0 + i < rows) __stcg(out + (r0 + i) * 128, __uint_as_float(g[i]));
          if (r0 + 8 + i < rows) __stcg(out + (r0 + 8 + i) * 128, __uint_as_float(h[i]));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty);
    }
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 128);
}

Args plan(const I8Stream& p, int sms) {
  Args a{};
  a.M = p.M;
  a.N = p.N;
  a.kb = (p.K + kStepK - 1) / kStepK;
  a.units = (p.N + 127) / 128;
  a.block_rows = p.M < kRows ? p.M : kRows;
  const int blocks = (p.M + kRows - 1) / kRows;
  a.chunks = plan_chunks(a.units, blocks, a.kb, a.block_rows, sms);
  a.items = blocks * a.units * a.chunks;
  a.n_cols = (a.block_rows + 15) / 16 * 16;
  a.raw_bytes = kRawW + a.n_cols * 128;
  a.op_bytes = kOpW + a.n_cols * 256;
  const int fit = (kSmemMax - 2048 - 2 * a.op_bytes) / a.raw_bytes;
  a.stages = fit < kMaxStages ? fit : kMaxStages;
  return a;
}

}  // namespace

StreamParts i8_stream_parts(const I8Stream& p, int sms) {
  const Args a = plan(p, sms);
  return StreamParts{nullptr, a.chunks, a.units, a.block_rows,
                     4 * static_cast<size_t>(a.items) * a.block_rows * 128, kRows};
}

int i8_stream(const I8Stream& p, const StreamParts& parts, const LoraDevice& d, bool early,
              cudaStream_t stream) {
  Args a = plan(p, d.sms);
  a.part = parts.part;
  a.wait_limit_ns = d.wait_limit_ns;
  a.status = d.status;
  CUtensorMap tmW{}, tmX{};
  if (int rc = encode_map_i8(&tmW, p.W, p.K, p.N, p.ldw, 128, kStepK)) return rc;
  if (int rc = encode_map_i8(&tmX, p.X, p.M, p.K, p.ldx, kStepK, a.n_cols)) return rc;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return GEMM_ERR_CUDA;
  static bool configured[64] = {};
  if (dev < 64 && !configured[dev]) {
    if (cudaFuncSetAttribute(i8_stream_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSmemMax) != cudaSuccess)
      return GEMM_ERR_CUDA;
    configured[dev] = true;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.items < d.sms ? a.items : d.sms), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = 2 * static_cast<size_t>(a.op_bytes) +
                         static_cast<size_t>(a.stages) * a.raw_bytes + 2048;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = early ? 1 : 0;
  return counted_launch(cudaLaunchKernelEx(&cfg, i8_stream_kernel, tmW, tmX, a)) == cudaSuccess
             ? GEMM_OK
             : GEMM_ERR_CUDA;
}

}  // namespace gb300
