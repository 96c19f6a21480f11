// lora_stream.cu -- the adapter product (and dX) where whole output tiles would
// leave SMs idle: a few rows (decoding), where the time is that of streaming W
// and the adapters from HBM once, and small outputs with a long K.
//
//   (lora_rows.cu)       V = s X A by (row, K slice) on CUDA cores
//   row_stream_kernel    X W as fp32 partial sums by (256 rows, 128 columns, K
//                        chunk): W is the M operand of tcgen05.mma, the rows of
//                        X the N operand, both by TMA.  It does not depend on
//                        the shrink, which runs beside it on the same SMs
//                        (programmatic launch).
//   lora_combine_kernel  C = alpha (sum of the chunks + V B[a]) + beta C, the
//                        chunks in k order, everything fp32, one rounding
//
// The low-rank product stays on CUDA cores here: each row has its own B[a], so
// on the tensor cores it would be 128 rows of zeros per adapter for 2 R
// multiply-adds per output that hide behind the loads of B anyway.
//
// Summing the chunks in a kernel of its own spreads that over all SMs: as K
// slices of the pair kernel, added up by the last to finish, 1000 x 1001 x 4096
// took 55 us instead of 31.  What bounds: at 64 x 4096 x 4096 W streams in 10.5
// of 15.6 us (34 MB, 0.48 of the measured HBM rate over its whole launch), the
// rest is the chain of three kernels; at one row the chain is all.
//
// Shared memory per ring stage: two 64-column boxes of 64 k-rows of W (128-byte
// swizzle, MN-major: LBO 8 KB, SBO 1 KB; or, for a W stored transposed, two
// boxes of 64 rows, K-major, SBO 1 KB), then the rows of X, 64 halves of k each
// (K-major, SBO 1 KB).
#include <type_traits>

#include "lora.h"

namespace gb300 {
namespace {

// ------------------------------------------------------------------- stream
constexpr int kWBytes = 2 * 64 * 128;       // 128 columns of a k-block of W
constexpr int kMaxStages = 12;
constexpr int kEpi = 4;
constexpr int kStreamThreads = 32 * (2 + kEpi);
constexpr int kBlockRows = 256;             // rows of an item (N of the MMA)
constexpr int kFewRows = 128;               // rows of a decoding batch
constexpr int kSmemMax = 232448;

struct CombineArgs {
  const float *part, *V;   // V: [row][slice][ldv]
  const uint16_t* F;       // F[a]: R x N, or N x R
  const int* ids;
  uint16_t* C;
  long long ldf, f_stride, ldc;
  int M, N, R, ldv, adapters, chunks, slices, units, block_rows;
  float alpha, beta;
  bool vec_c;              // rows of C on the 8-byte grid
};

struct StreamArgs {
  int M, N, trans;
  int kb, chunks, units, items;   // k-blocks, chunks, 128-column units, blocks x units x chunks
  int stages, stage_bytes, n_cols, acc_cols;
  int block_rows;          // rows of a block's partial sums: min(M, kBlockRows)
  float* part;             // [block][unit][chunk][row][128]
  unsigned long long wait_limit_ns;
  DeviceStatus* status;
};

__global__ void __launch_bounds__(kStreamThreads, 1)
    row_stream_kernel(const __grid_constant__ CUtensorMap tmW,
                      const __grid_constant__ CUtensorMap tmX, const StreamArgs p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const base_ptr = smem_raw + (base - raw);
  const int S = p.stages;
  const int warp = warp_id_uniform(), lane = static_cast<int>(lane_id());
  const uint32_t bars = base + static_cast<uint32_t>(S * p.stage_bytes);
  auto full_bar = [&](int s) { return bars + 8u * s; };
  auto empty_bar = [&](int s) { return bars + 8u * (kMaxStages + s); };
  auto accf_bar = [&](uint32_t b) { return bars + 8u * (2 * kMaxStages + b); };
  auto acce_bar = [&](uint32_t b) { return bars + 8u * (2 * kMaxStages + 2 + b); };
  const uint32_t done_bar = bars + 8u * (2 * kMaxStages + 4);
  constexpr int kBars = 2 * kMaxStages + 5;
  uint8_t* const tmem_ptr = base_ptr + static_cast<size_t>(S) * p.stage_bytes + 8 * kBars;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1u);
      mbar_init(empty_bar(s), 1u);
    }
    for (uint32_t b = 0; b < 2; ++b) {
      mbar_init(accf_bar(b), 1u);
      mbar_init(acce_bar(b), static_cast<uint32_t>(kEpi));
    }
    mbar_init(done_bar, 1u);
    fence_barrier_init();
    fence_proxy_async_smem();
    prefetch_tensormap(&tmW);
    prefetch_tensormap(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(tmem_ptr), 2 * p.acc_cols);
    tmem_relinquish();
    // only now: a kernel after the next one (the sums) allocates tensor memory and
    // holds it until this one ends
    griddep_launch_dependents();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_ptr);
  const unsigned long long limit = p.wait_limit_ns;
  DeviceStatus* const st = p.status;

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t policy = l2_evict_first_policy();
      int stage = 0;
      uint32_t phase = 0, issued = 0;
      bool ok = true;
      for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
        const int c = it % p.chunks, n0 = it / p.chunks % p.units * 128;
        const int row0 = it / p.chunks / p.units * kBlockRows;
        const bool two = n0 + 64 < p.N;      // the second box lies in the matrix
        const uint32_t bytes =
            static_cast<uint32_t>((two ? kWBytes : kWBytes / 2) + p.n_cols * 128);
        for (int kb = c * p.kb / p.chunks; kb < (c + 1) * p.kb / p.chunks; ++kb) {
          if (!wait_parity(empty_bar(stage), phase ^ 1u, limit, st, 60)) {
            ok = false;
            break;
          }
          const uint32_t dst = base + static_cast<uint32_t>(stage * p.stage_bytes);
          mbar_arrive_expect_tx(full_bar(stage), bytes);
          // W evict-first when no other block of rows reads it
          for (int b = 0; b <= two; ++b) {
            const int n = n0 + 64 * b, cx = p.trans ? kb * 64 : n, cy = p.trans ? n : kb * 64;
            if (p.M <= kBlockRows)
              tma_load_2d_hint(dst + b * 8192, &tmW, full_bar(stage), cx, cy, policy);
            else
              tma_load_2d(dst + b * 8192, &tmW, full_bar(stage), cx, cy);
          }
          tma_load_2d(dst + kWBytes, &tmX, full_bar(stage), kb * 64, row0);
          ++issued;
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      const uint32_t n = min(issued, static_cast<uint32_t>(S));
      for (uint32_t i = issued - n; i < issued; ++i)
        settle_wait(full_bar(static_cast<int>(i % S)), (i / S) & 1u, st, 61);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc =
          make_idesc(0u, 128u, static_cast<uint32_t>(p.n_cols), p.trans ? 0u : 1u, 0u);
      int stage = 0;
      uint32_t phase = 0, local = 0;
      bool ok = true;
      for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
        const int c = it % p.chunks;
        const int kb0 = c * p.kb / p.chunks, kb1 = (c + 1) * p.kb / p.chunks;
        const uint32_t buf = local & 1u;
        if (!wait_parity(acce_bar(buf), ((local >> 1) & 1u) ^ 1u, limit, st, 62)) break;
        tc_fence_after();
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!wait_parity(full_bar(stage), phase, limit, st, 63)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t w0 = base + static_cast<uint32_t>(stage * p.stage_bytes);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_f16_ss(tmem + buf * p.acc_cols,
                       p.trans ? smem_desc_sw128(w0 + kk * 32, 16u, 1024u)
                               : smem_desc_sw128(w0 + kk * 2048, 8192u, 1024u),
                       smem_desc_sw128(w0 + kWBytes + kk * 32, 16u, 1024u), idesc,
                       (kb > kb0 || kk > 0) ? 1u : 0u);
          mma_commit(empty_bar(stage));
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        mma_commit(accf_bar(buf));
        ++local;
      }
      mma_commit(done_bar);
      settle_wait(done_bar, 0u, st, 64);
    }
    __syncwarp();
  } else {
    const int quad = warp & 3;
    uint32_t local = 0;
    for (int it = blockIdx.x; it < p.items; it += gridDim.x, ++local) {
      const uint32_t buf = local & 1u;
      if (!wait_parity(accf_bar(buf), (local >> 1) & 1u, limit, st, 65)) break;
      tc_fence_after();
      const uint32_t d0 = tmem + (static_cast<uint32_t>(32 * quad) << 16) + buf * p.acc_cols;
      float* const out =
          p.part + static_cast<long long>(it) * p.block_rows * 128 + 32 * quad + lane;
      const int rows = min(kBlockRows, p.M - it / p.chunks / p.units * kBlockRows);
      for (int r0 = 0; r0 < rows; r0 += 16) {   // n_cols is a multiple of 16
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
      if (lane == 0) mbar_arrive(acce_bar(buf));
    }
    // this kernel's end stands for the shrink's too (the combine waits for it)
    griddep_wait();
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 2 * p.acc_cols);
}

// ------------------------------------------------------------------ combine
constexpr int kCombThreads = 128;

// Few rows: one block per (row, 128 VEC columns), VEC columns a thread (four
// when that still fills the SMs; a thread then takes them with one load).  All
// that it waits for are three rounds of loads -- the id, then the first ranks of
// F[a] (which no kernel before it writes), then V's slices and the chunks
// together -- and little code: with everything unrolled, 2048 columns of one row
// took 13 us here instead of 6.
constexpr int kAhead = 16;

template <bool TRANS, int VEC>
__global__ void __launch_bounds__(kCombThreads) lora_combine_row_kernel(const CombineArgs p) {
  static_assert(VEC == 1 || (VEC == 4 && !TRANS), "four columns are one load along a row of F");
  __shared__ float raw[kLoraRowSlices * kLoraMaxRank];
  __shared__ float vs[kLoraMaxRank];
  griddep_launch_dependents();
  const int strips = (p.N + kCombThreads * VEC - 1) / (kCombThreads * VEC);
  const int i = blockIdx.x / strips;
  const int t = threadIdx.x, c = ((blockIdx.x - i * strips) * kCombThreads + t) * VEC;
  const int a = __ldg(p.ids + i);
  const bool has = a >= 0 && a < p.adapters, mine = has && c < p.N;
  const uint16_t* const f =
      p.F + (mine ? a * p.f_stride + (TRANS ? static_cast<long long>(c) * p.ldf : c) : 0);
  const long long step = p.ldf;
  const bool whole = c + VEC <= p.N;
  // ranks r .. r + 7 of this thread's column (TRANS): one load where they are there
  auto load8 = [&](int r, uint16_t (&w)[8]) {
    if (r + 8 <= p.R) {
      const uint4 q = __ldg(reinterpret_cast<const uint4*>(f + r));
      memcpy(w, &q, sizeof(w));
    } else {
#pragma unroll
      for (int u = 0; u < 8; ++u) w[u] = r + u < p.R ? __ldg(f + r + u) : 0;
    }
  };
  auto load = [&](int r, uint16_t (&w)[VEC]) {
    if (VEC == 4 && whole) {
      const uint2 q = __ldg(reinterpret_cast<const uint2*>(f + r * step));
      memcpy(w, &q, sizeof(w));
    } else {
#pragma unroll
      for (int u = 0; u < VEC; ++u) w[u] = c + u < p.N ? __ldg(f + r * step + u) : 0;
    }
  };
  uint16_t b[kAhead][VEC];
  if (mine) {
    if (TRANS) {
#pragma unroll
      for (int r = 0; r < kAhead; r += 8)
        if (r < p.R) {
          uint16_t w[8];
          load8(r, w);
#pragma unroll
          for (int u = 0; u < 8; ++u) b[r + u][0] = w[u];
        }
    } else {
#pragma unroll
      for (int r = 0; r < kAhead; ++r)
        if (r < p.R) load(r, b[r]);
    }
  }
  griddep_wait();
  if (has) {
    const float* const v = p.V + static_cast<long long>(i) * p.slices * p.ldv;
    for (int e = t; e < p.slices * p.ldv; e += kCombThreads) raw[e] = __ldcg(v + e);
  }
  const long long chunk_elems = static_cast<long long>(p.block_rows) * 128;
  const int blk = i / kBlockRows;
  const float* const part =
      p.part +
      (static_cast<long long>(blk) * p.units + min(c >> 7, p.units - 1)) * p.chunks * chunk_elems +
      (i - blk * kBlockRows) * 128 + (c & 127);
  float s[VEC] = {};
#pragma unroll 4
  for (int k = 0; k < p.chunks; ++k) {
    if (VEC == 4) {
      const float4 q = __ldcg(reinterpret_cast<const float4*>(part + k * chunk_elems));
      s[0] += q.x;
      s[VEC > 1 ? 1 : 0] += VEC > 1 ? q.y : 0.0f;
      s[VEC > 2 ? 2 : 0] += VEC > 2 ? q.z : 0.0f;
      s[VEC > 3 ? 3 : 0] += VEC > 3 ? q.w : 0.0f;
    } else {
      s[0] += __ldcg(part + k * chunk_elems);
    }
  }
  __syncthreads();
  if (has && t < p.R) {
    float x = 0.0f;
    for (int k = 0; k < p.slices; ++k) x += raw[k * p.ldv + t];
    vs[t] = x;
  }
  __syncthreads();
  if (c >= p.N) return;
  if (has) {
    float l[VEC] = {};
#pragma unroll
    for (int r = 0; r < kAhead; ++r)
      if (r < p.R)
#pragma unroll
        for (int u = 0; u < VEC; ++u) l[u] = fmaf(vs[r], lora_h2f(b[r][u]), l[u]);
    if (TRANS) {
#pragma unroll 2
      for (int r = kAhead; r < p.R; r += 8) {
        uint16_t w[8];
        load8(r, w);
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (r + u < p.R) l[0] = fmaf(vs[r + u], lora_h2f(w[u]), l[0]);
      }
    } else {
#pragma unroll 4
      for (int r = kAhead; r < p.R; ++r) {
        uint16_t w[VEC];
        load(r, w);
#pragma unroll
        for (int u = 0; u < VEC; ++u) l[u] = fmaf(vs[r], lora_h2f(w[u]), l[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < VEC; ++u) s[u] += l[u];
  }
  uint16_t* const dst = p.C + static_cast<long long>(i) * p.ldc + c;
  uint16_t h[VEC];
#pragma unroll
  for (int u = 0; u < VEC; ++u)
    if (c + u < p.N)
      h[u] = lora_f2h(p.beta != 0.0f ? fmaf(p.alpha, s[u], p.beta * lora_h2f(dst[u])) : p.alpha * s[u]);
  if (VEC == 4 && whole && p.vec_c) {
    uint2 q;
    memcpy(&q, h, sizeof(q));
    *reinterpret_cast<uint2*>(dst) = q;
  } else {
#pragma unroll
    for (int u = 0; u < VEC; ++u)
      if (c + u < p.N) dst[u] = h[u];
  }
}

// More rows: one block per (RB rows, 512 columns), four columns a thread.  Rows of one
// adapter share the loads of F[a] (the rows of a prompt do; row by row, 1500 x
// 1000 outputs of rank 24 read 72 MB of it from L2 and took 26 us).
template <bool TRANS, int RB>
__global__ void __launch_bounds__(kCombThreads) lora_combine_kernel(const CombineArgs p) {
  __shared__ __align__(16) float vs[RB][kLoraMaxRank];
  griddep_launch_dependents();
  const int strips = (p.N + 4 * kCombThreads - 1) / (4 * kCombThreads);
  const int i0 = blockIdx.x / strips * RB;
  const int c = blockIdx.x % strips * 4 * kCombThreads + 4 * static_cast<int>(threadIdx.x);
  const bool whole = c + 4 <= p.N;
  int id[RB];
#pragma unroll
  for (int j = 0; j < RB; ++j) {
    id[j] = i0 + j < p.M ? __ldg(p.ids + i0 + j) : -1;
    if (id[j] >= p.adapters) id[j] = -1;
  }
  const long long f0 = TRANS ? static_cast<long long>(c) * p.ldf : c;
  // nothing of the kernels before this one is read yet: bring this block's
  // part of the first row's F[a] into L2
  if (id[0] >= 0 && c < p.N) {
    const uint16_t* const f = p.F + id[0] * p.f_stride + f0;
    if (TRANS) {
      for (int j = 0; j < 4 && c + j < p.N; ++j) prefetch_l2(f + j * p.ldf);
    } else if ((threadIdx.x & 15) == 0) {
      for (int r = 0; r < p.R; ++r) prefetch_l2(f + r * p.ldf);
    }
  }
  griddep_wait();
  // V by 16-byte pieces (one slice), the ranks past R up to a multiple of four
  // with it (they are zero)
  const int per = p.ldv / 4;
#pragma unroll 4
  for (int e = threadIdx.x; e < RB * per; e += kCombThreads) {
    const int j = e / per, r = (e - j * per) * 4;
    const int row = min(i0 + j, p.M - 1);
    *reinterpret_cast<float4*>(&vs[j][r]) =
        __ldcg(reinterpret_cast<const float4*>(p.V + static_cast<long long>(row) * p.ldv + r));
  }
  __syncthreads();
  if (c >= p.N) return;
  const long long chunk_elems = static_cast<long long>(p.block_rows) * 128;
  const int blk = i0 / kBlockRows;   // RB divides kBlockRows
  const float* const part =
      p.part + (static_cast<long long>(blk) * p.units + (c >> 7)) * p.chunks * chunk_elems +
      (i0 - blk * kBlockRows) * 128 + (c & 127);
  float o[RB][4];
#pragma unroll
  for (int j = 0; j < RB; ++j)
#pragma unroll
    for (int u = 0; u < 4; ++u) o[j][u] = 0.0f;
#pragma unroll 2
  for (int k = 0; k < p.chunks; ++k)
#pragma unroll
    for (int j = 0; j < RB; ++j)
      if (i0 + j < p.M) {
        const float4 t = __ldcg(reinterpret_cast<const float4*>(part + k * chunk_elems + j * 128));
        o[j][0] += t.x;
        o[j][1] += t.y;
        o[j][2] += t.z;
        o[j][3] += t.w;
      }
  unsigned int todo = 0;
#pragma unroll
  for (int j = 0; j < RB; ++j) todo |= static_cast<unsigned int>(id[j] >= 0) << j;
  while (todo) {
    int a = -1;
    unsigned int mine = 0;   // the rows of the first open row's adapter
#pragma unroll
    for (int j = 0; j < RB; ++j)
      if (todo >> j & 1u) {
        if (a < 0) a = id[j];
        if (id[j] == a) mine |= 1u << j;
      }
    todo &= ~mine;
    const uint16_t* const f = p.F + a * p.f_stride + f0;
    // four ranks at a time: w[k][u] is rank r + k of column c + u; a row's four
    // entries of V are one load from shared memory
    auto add4 = [&](int r, const float (&w)[4][4]) {
#pragma unroll
      for (int j = 0; j < RB; ++j)
        if (mine >> j & 1u) {
          const float4 v = *reinterpret_cast<const float4*>(&vs[j][r]);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            o[j][u] = fmaf(v.x, w[0][u], o[j][u]);
            o[j][u] = fmaf(v.y, w[1][u], o[j][u]);
            o[j][u] = fmaf(v.z, w[2][u], o[j][u]);
            o[j][u] = fmaf(v.w, w[3][u], o[j][u]);
          }
        }
    };
    int r = 0;
    if (TRANS) {
#pragma unroll 2
      for (; r + 8 <= p.R; r += 8) {
        uint4 q[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          q[u] = __ldg(reinterpret_cast<const uint4*>(f + (c + u < p.N ? u * p.ldf : 0) + r));
        float w[4][4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float2 b0 = lora_h2f2(q[u].x), b1 = lora_h2f2(q[u].y);
          w[0][u] = b0.x; w[1][u] = b0.y; w[2][u] = b1.x; w[3][u] = b1.y;
        }
        add4(r, w);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float2 b0 = lora_h2f2(q[u].z), b1 = lora_h2f2(q[u].w);
          w[0][u] = b0.x; w[1][u] = b0.y; w[2][u] = b1.x; w[3][u] = b1.y;
        }
        add4(r + 4, w);
      }
    } else if (whole) {
#pragma unroll 2
      for (; r + 4 <= p.R; r += 4) {
        uint2 q[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) q[k] = __ldg(reinterpret_cast<const uint2*>(f + (r + k) * p.ldf));
        float w[4][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 b0 = lora_h2f2(q[k].x), b1 = lora_h2f2(q[k].y);
          w[k][0] = b0.x; w[k][1] = b0.y; w[k][2] = b1.x; w[k][3] = b1.y;
        }
        add4(r, w);
      }
    }
    for (; r < p.R; r += 4) {   // the last ranks, the ragged last columns
      float w[4][4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int u = 0; u < 4; ++u)
          w[k][u] = c + u < p.N && r + k < p.R
                        ? lora_h2f(TRANS ? f[u * p.ldf + r + k] : f[(r + k) * p.ldf + u])
                        : 0.0f;
      add4(r, w);
    }
  }
#pragma unroll
  for (int j = 0; j < RB; ++j) {
    if (i0 + j >= p.M) break;
    uint16_t* const dst = p.C + static_cast<long long>(i0 + j) * p.ldc + c;
    if (whole && p.vec_c) {
      float2 old0 = make_float2(0.0f, 0.0f), old1 = old0;
      if (p.beta != 0.0f) {
        const uint2 b = *reinterpret_cast<const uint2*>(dst);
        old0 = lora_h2f2(b.x);
        old1 = lora_h2f2(b.y);
      }
      const float old[4] = {old0.x, old0.y, old1.x, old1.y};
      uint32_t h[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        h[u] = lora_f2h(p.beta != 0.0f ? fmaf(p.alpha, o[j][u], p.beta * old[u]) : p.alpha * o[j][u]);
      *reinterpret_cast<uint2*>(dst) = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (c + u < p.N)
          dst[u] = lora_f2h(p.beta != 0.0f ? fmaf(p.alpha, o[j][u], p.beta * lora_h2f(dst[u]))
                                           : p.alpha * o[j][u]);
    }
  }
}

// Chunks per unit: the count whose rounds of chunks over the SMs, in k-block
// times of an SM, and whose partial sums take least.  A k-block takes 0.36 us
// (its 16 KB of W at an SM's share of HBM) or, for a full block of rows, as long
// as its 48 KB from L2; the partial sums are 1 KB per row written and read,
// through L2 at about twice HBM's rate.
int plan_chunks(int units, int blocks, int kb, int rows, int sms) {
  int best = 1;
  double best_t = 1e30;
  for (int c = 1; c <= std::min(kb, 32); ++c) {
    const long long rounds = (1ll * units * blocks * c + sms - 1) / sms;
    const double t = static_cast<double>(rounds) * ((kb + c - 1) / c + 2) +
                     1.9e-4 * units * blocks * c * rows;
    if (t < best_t) {
      best_t = t;
      best = c;
    }
  }
  return best;
}

// K slices of the shrink: about four blocks per SM in all, at least 64 long; one
// where several rows of a block of the sum kernel can share an adapter.
int shrink_slices(const LoraStream& p, int sms) {
  return p.M > 2 * kFewRows ? 1
                            : std::max(1, std::min({kLoraRowSlices, 4 * sms / p.M, p.K / 64}));
}

StreamArgs plan(const LoraStream& p, int sms) {
  StreamArgs t{};
  t.M = p.M;
  t.N = p.N;
  t.trans = p.trans;
  t.kb = (p.K + 63) / 64;
  t.units = (p.N + 127) / 128;
  t.block_rows = std::min(p.M, kBlockRows);
  const int blocks = (p.M + kBlockRows - 1) / kBlockRows;
  t.chunks = plan_chunks(t.units, blocks, t.kb, t.block_rows, sms);
  t.items = blocks * t.units * t.chunks;
  t.n_cols = (t.block_rows + 15) / 16 * 16;
  t.acc_cols = t.n_cols > 128 ? 256 : 128;
  t.stage_bytes = kWBytes + t.n_cols * 128;
  // beside the blocks of the shrink by rows (10 KB each, four on an SM) where it
  // runs: with the whole shared memory this kernel's CTAs started only as those
  // ended, 3 us later
  t.stages = std::min(kMaxStages, ((p.V ? kSmemMax : kSmemMax - 49152) - 2048) / t.stage_bytes);
  return t;
}

}  // namespace

bool lora_stream_suits(int M, int N, int sms) {
  const long long tiles = static_cast<long long>((M + 255) / 256) * ((N + 255) / 256);
  return M <= kFewRows || 4 * tiles <= sms;
}

// By rows: each row's adapter is read from L2 by itself, 2 K R bytes, whatever
// the other rows have: 10 us for 2^25 multiply-adds, what the tensor cores take
// with a few adapters among 128 rows; with many they make many passes (300 rows
// of 4096 over 32 adapters of rank 16 in no order: 70 us).  Up to 128 rows by rows
// whatever K R is: a call of 128 x 4096 x 8192 at rank 128 takes 69 us with one
// adapter (43 with the tensor cores) and 110 with 32 in no order (272), one of
// 128 x 4096 x 4096 at rank 16 17 us with either (17 and 81).  How many adapters
// there are only the device knows.
bool lora_stream_shrinks(int M, int K, int R) {
  return M <= kFewRows || (M <= 4 * kFewRows && 1ll * M * K * R <= (1ll << 25));
}

size_t lora_stream_bytes(const LoraStream& p, int sms) {
  const StreamArgs t = plan(p, sms);
  const size_t v = p.V ? 0 : 4 * static_cast<size_t>(p.M) * shrink_slices(p, sms) * ((p.R + 7) / 8 * 8);
  return lora_round256(v) + 4 * static_cast<size_t>(t.items) * t.block_rows * 128;
}

int lora_stream(const LoraStream& p, void* scratch, const LoraDevice& d, cudaStream_t stream) {
  StreamArgs t = plan(p, d.sms);
  CUtensorMap tmW{}, tmX{};
  if (int rc = p.trans ? encode_map_f16(&tmW, p.W, p.N, p.K, p.ldw, 64, 64)
                       : encode_map_f16(&tmW, p.W, p.K, p.N, p.ldw, 64, 64))
    return rc;
  if (int rc = encode_map_f16(&tmX, p.X, p.M, p.K, p.ldx, 64, t.n_cols)) return rc;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return GEMM_ERR_CUDA;
  static bool configured[64] = {};
  if (dev < 64 && !configured[dev]) {
    if (cudaFuncSetAttribute(row_stream_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSmemMax) != cudaSuccess)
      return GEMM_ERR_CUDA;
    configured[dev] = true;
  }
  t.wait_limit_ns = d.wait_limit_ns;
  t.status = d.status;
  CombineArgs c{};
  c.V = p.V;
  c.ldv = p.ldv;
  c.slices = 1;
  uint8_t* rest = static_cast<uint8_t*>(scratch);
  if (!p.V) {
    const int slices = shrink_slices(p, d.sms), r8 = (p.R + 7) / 8 * 8;
    float* const v = reinterpret_cast<float*>(rest);
    rest += lora_round256(4 * static_cast<size_t>(p.M) * slices * r8);
    LoraRows rows{};
    rows.job[0] = LoraRowsJob{p.X, p.ldx, p.K, p.A, p.lda, p.a_stride, 0, v, p.R};
    rows.njobs = 1;
    rows.slices = slices;
    rows.ids = p.ids;
    rows.scales = p.scales;
    rows.M = p.M;
    rows.R = r8;
    rows.adapters = p.adapters;
    if (launch_lora_rows(rows, stream) != cudaSuccess) return GEMM_ERR_CUDA;
    c.V = v;
    c.ldv = r8;
    c.slices = slices;
  }
  t.part = reinterpret_cast<float*>(rest);
  c.part = t.part;
  c.F = p.F;
  c.ids = p.ids;
  c.C = p.C;
  c.ldf = p.ldf;
  c.f_stride = p.f_stride;
  c.ldc = p.ldc;
  c.M = p.M;
  c.N = p.N;
  c.R = p.R;
  c.adapters = p.adapters;
  c.chunks = t.chunks;
  c.units = t.units;
  c.block_rows = t.block_rows;
  c.alpha = p.alpha;
  c.beta = p.beta;
  c.vec_c = (reinterpret_cast<uintptr_t>(p.C) & 7u) == 0 && p.ldc % 4 == 0;

  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min(t.items, d.sms)), 1, 1);
  cfg.blockDim = dim3(kStreamThreads, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(t.stages) * t.stage_bytes + 2048;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (counted_launch(cudaLaunchKernelEx(&cfg, row_stream_kernel, tmW, tmX, t)) != cudaSuccess)
    return GEMM_ERR_CUDA;

  // as many rows a block as leave a few blocks per SM; else by single rows
  const long long strips = (p.N + 4 * kCombThreads - 1) / (4 * kCombThreads);
  const int rb = c.slices > 1                     ? 1
                 : p.M * strips >= 16ll * d.sms ? 8
                 : p.M * strips >= 8ll * d.sms  ? 4
                                                : 1;
  const bool wide = !p.trans && p.M * strips >= d.sms;   // four columns a thread
  const long long blocks = rb > 1 ? (p.M + rb - 1) / rb * strips : p.M * (wide ? strips : t.units);
  if (blocks > 0x7fffffff) return GEMM_ERR_ARG;
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
  cfg.blockDim = dim3(kCombThreads, 1, 1);
  cfg.dynamicSmemBytes = 0;
  auto launch = [&](auto trans) {
    constexpr bool T = decltype(trans)::value;
    return rb == 8   ? cudaLaunchKernelEx(&cfg, lora_combine_kernel<T, 8>, c)
           : rb == 4 ? cudaLaunchKernelEx(&cfg, lora_combine_kernel<T, 4>, c)
                     : wide    ? cudaLaunchKernelEx(&cfg, lora_combine_row_kernel<false, 4>, c)
                     : cudaLaunchKernelEx(&cfg, lora_combine_row_kernel<T, 1>, c);
  };
  const cudaError_t e = p.trans ? launch(std::true_type{}) : launch(std::false_type{});
  return counted_launch(e) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

}  // namespace gb300
