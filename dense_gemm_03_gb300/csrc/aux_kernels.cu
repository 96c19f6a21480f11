// aux_kernels.cu -- HBM-bound helper kernels of the GEMM path:
//   * split-K reduction: C = half(alpha * sum_s P_s + beta * C), slices summed
//     in ascending order (deterministic), fp32 arithmetic, one rounding;
//   * realignment of an operand whose rows are not 16-byte aligned into an
//     aligned copy, so that the tensor-core kernel can load it by TMA, and the
//     copy of such a C back from the aligned copy the kernel wrote by TMA;
//   * the big/small tf32 split of fp32 operands for the 3xTF32 SGEMM, and the
//     scaled two-part fp16 split for the 3xFP16 SGEMM;
//   * scale-only update for alpha == 0 or K == 0: C := beta*C (C := 0 when
//     beta == 0, without reading C -- the convention of the "LeetGPU GEMM T4"
//     WMMA sections and the "advanced SGEMM" page for beta == 0).
// Grid-stride loops over rows x column groups; 4-wide vectors where the
// row stride and the base pointer allow it.
#include <cuda_fp16.h>

#include "internal.h"
#include "ptx.cuh"

namespace gb300 {
namespace {

__device__ __forceinline__ float half_bits_to_float(uint16_t b) {
  return __half2float(__ushort_as_half(b));
}
__device__ __forceinline__ uint16_t float_to_half_bits(float x) {
  return __half_as_ushort(__float2half_rn(x));
}

// One thread per group of 4 consecutive columns of one row.
__global__ void splitk_reduce_f16_kernel(const float* __restrict__ ws, long long ws_ld, int splits,
                                         uint16_t* __restrict__ C, long long ldc, int M, int N,
                                         float alpha, float beta) {
  const int groups = (N + 3) >> 2;
  const long long total = static_cast<long long>(M) * groups;
  const long long slice = static_cast<long long>(M) * ws_ld;
  const bool has_c = beta != 0.0f;
  for (long long g = blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x; g < total;
       g += static_cast<long long>(gridDim.x) * blockDim.x) {
    const int row = static_cast<int>(g / groups);
    const int col = static_cast<int>(g % groups) * 4;
    const float* w = ws + static_cast<long long>(row) * ws_ld + col;
    float4 s = *reinterpret_cast<const float4*>(w);   // ws_ld % 4 == 0, 16-byte aligned
    for (int k = 1; k < splits; ++k) {
      const float4 v = *reinterpret_cast<const float4*>(w + k * slice);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    const float acc[4] = {s.x, s.y, s.z, s.w};
    uint16_t* c = C + static_cast<long long>(row) * ldc + col;
    const int n = min(4, N - col);
    for (int i = 0; i < n; ++i) {
      const float o = has_c ? __fmaf_rn(alpha, acc[i], beta * half_bits_to_float(c[i]))
                            : alpha * acc[i];
      c[i] = float_to_half_bits(o);
    }
  }
}

__global__ void scale_f16_kernel(uint16_t* __restrict__ C, long long ldc, int M, int N,
                                 float beta) {
  const long long total = static_cast<long long>(M) * N;
  for (long long i = blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * blockDim.x) {
    const int row = static_cast<int>(i / N), col = static_cast<int>(i % N);
    uint16_t* c = C + static_cast<long long>(row) * ldc + col;
    *c = (beta == 0.0f) ? float_to_half_bits(0.0f) : float_to_half_bits(beta * half_bits_to_float(*c));
  }
}

__global__ void scale_f32_kernel(float* __restrict__ C, long long ldc, int M, int N, float beta) {
  const long long total = static_cast<long long>(M) * N;
  for (long long i = blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * blockDim.x) {
    const int row = static_cast<int>(i / N), col = static_cast<int>(i % N);
    float* c = C + static_cast<long long>(row) * ldc + col;
    *c = (beta == 0.0f) ? 0.0f : beta * *c;
  }
}

// 16 bytes starting `m` bytes (m even, 2..14) into the 32 bytes lo|hi.
__device__ __forceinline__ uint4 shift_bytes(uint4 lo, uint4 hi, uint32_t m) {
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  const uint32_t sh = (m & 3u) * 8u;
  uint32_t o[4];
  switch (m >> 2) {
#define GB300_SEL(Q)                                                          \
  case Q:                                                                     \
    for (int i = 0; i < 4; ++i) o[i] = __funnelshift_r(w[Q + i], w[Q + i + 1], sh); \
    break;
    GB300_SEL(0)
    GB300_SEL(1)
    GB300_SEL(2)
    default:
      for (int i = 0; i < 4; ++i) o[i] = __funnelshift_r(w[3 + i], w[4 + i], sh);
      break;
#undef GB300_SEL
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// dst[r][c] = src[r][c] for c < cols, 0 for cols <= c < width (width % 8 == 0,
// dst 16-byte aligned).  One thread writes 8 halves.  A fully valid source
// piece at any 2-byte alignment is read as the (at most two) 16-byte-aligned
// blocks that contain it -- blocks that hold at least one element of the
// piece, so the reads never leave memory the caller owns -- and shifted into
// place; the ragged end of a row uses element loads.
__device__ __forceinline__ void realign_rows(const uint16_t* __restrict__ src, long long lds,
                                             uint16_t* __restrict__ dst, long long ldd, int rows,
                                             int cols, long long width, long long block,
                                             long long nblocks) {
  const long long groups = width / 8;
  const long long total = static_cast<long long>(rows) * groups;
  for (long long g = block * blockDim.x + threadIdx.x; g < total; g += nblocks * blockDim.x) {
    const int r = static_cast<int>(g / groups);
    const int c0 = static_cast<int>(g % groups) * 8;
    const uint16_t* p = src + static_cast<long long>(r) * lds + c0;
    uint4 v;
    if (c0 + 8 <= cols) {
      const uintptr_t a = reinterpret_cast<uintptr_t>(p);
      const uint32_t m = static_cast<uint32_t>(a & 15u);
      const uint4* blk = reinterpret_cast<const uint4*>(a - m);
      // m is even: half pointers are 2-byte aligned (checked by the host).
      // blk + 1 starts 16 - m bytes into the 16 bytes read, so both aligned
      // blocks hold bytes of the row: no read leaves a 16-byte block (and so
      // a page) that holds operand data.
      v = (m == 0) ? __ldg(blk) : shift_bytes(__ldg(blk), __ldg(blk + 1), m);
    } else {
      uint32_t h[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = (c0 + i < cols) ? static_cast<uint32_t>(__ldg(p + i)) : 0u;
      v = make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16),
                     h[6] | (h[7] << 16));
    }
    *reinterpret_cast<uint4*>(dst + static_cast<long long>(r) * ldd + c0) = v;
  }
}

// Several copies in one launch: blocks [end[i-1], end[i]) copy job i.
__global__ void realign_f16_kernel(const RealignBatch b) {
  griddep_wait();
  int i = 0;
  while (i + 1 < b.n && static_cast<int>(blockIdx.x) >= b.end[i]) ++i;
  const int first = i ? b.end[i - 1] : 0;
  const RealignJob& j = b.job[i];
  realign_rows(j.src, j.lds, j.dst, j.ldd, j.rows, j.cols, j.width ? j.width : j.ldd,
               blockIdx.x - first, b.end[i] - first);
  // this block's copies are issued: the GEMM launched next may be scheduled
  // (it waits for this kernel's completion before reading the copies)
  griddep_launch_dependents();
}

// dst[r][c] := src[r][c] for c < cols; src rows 16-byte aligned with
// lds >= cols rounded up to 8, dst rows at any 2-byte alignment.  One thread
// writes one 16-byte-aligned piece of a destination row, so that a warp's
// stores are contiguous: a piece inside the row's columns with one 16-byte
// store (its 8 halves read as the two aligned 16-byte blocks of the source
// row that hold them, which lie within the row's lds, and shifted into
// place), the pieces at the two ends of the row element by element (nothing
// outside the row's columns is written).
__device__ __forceinline__ void unalign_rows(const uint16_t* __restrict__ src, long long lds,
                                             uint16_t* __restrict__ dst, long long ldd, int rows,
                                             int cols, long long block, long long nblocks) {
  const long long pieces = cols / 8 + 2;   // enough for any alignment of a row
  const long long total = static_cast<long long>(rows) * pieces;
  for (long long g = block * blockDim.x + threadIdx.x; g < total; g += nblocks * blockDim.x) {
    const int r = static_cast<int>(g / pieces);
    const int j = static_cast<int>(g % pieces);
    uint16_t* const d = dst + static_cast<long long>(r) * ldd;
    const int md = static_cast<int>(reinterpret_cast<uintptr_t>(d) & 15u);   // even
    const int e0 = 8 * j - md / 2;   // first element of the row in piece j
    if (e0 >= cols) continue;
    const uint16_t* const s = src + static_cast<long long>(r) * lds;
    if (e0 >= 0 && e0 + 8 <= cols) {
      const uint4* const blk = reinterpret_cast<const uint4*>(s + (e0 & ~7));
      const uint32_t m = static_cast<uint32_t>(e0 & 7) * 2u;
      const uint4 v = (m == 0) ? __ldg(blk) : shift_bytes(__ldg(blk), __ldg(blk + 1), m);
      __stcs(reinterpret_cast<uint4*>(d + e0), v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = e0 + i;
        if (e >= 0 && e < cols) d[e] = __ldg(s + e);
      }
    }
  }
}

__global__ void unalign_f16_kernel(const RealignBatch b) {
  griddep_wait();   // the kernel that writes the sources may still be running
  int i = 0;
  while (i + 1 < b.n && static_cast<int>(blockIdx.x) >= b.end[i]) ++i;
  const int first = i ? b.end[i - 1] : 0;
  const RealignJob& j = b.job[i];
  unalign_rows(j.src, j.lds, j.dst, j.ldd, j.rows, j.cols, blockIdx.x - first, b.end[i] - first);
}

// tf32 value nearest to x (ties away from zero), as fp32 bits with the low 13
// bits clear.
__device__ __forceinline__ float round_tf32(float x) {
  uint32_t r;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
  return __uint_as_float(r);
}

// big = x with the low 13 mantissa bits cleared (exactly representable in
// tf32), small = tf32(x - big); x = big + small up to about 2^-22 |x|.
// Non-finite x: big carries it, small = 0.
__device__ __forceinline__ void split_tf32(float x, float& big, float& small) {
  const uint32_t bits = __float_as_uint(x);
  if (isnan(x)) {
    big = __uint_as_float(0x7FFFE000u);
    small = 0.0f;
  } else if (isinf(x)) {
    big = x;
    small = 0.0f;
  } else {
    big = __uint_as_float(bits & 0xFFFFE000u);
    small = round_tf32(x - big);
  }
}

// Splits a rows x cols fp32 matrix (any leading dimension, 4-byte aligned)
// into big and small parts stored densely with leading dimension ldd
// (ldd % 4 == 0, zero padding), one thread per 4 output columns; `block` and
// `nblocks` number the blocks that share the work.
__device__ __forceinline__ void split_rows(const float* __restrict__ src, long long lds,
                                           float* __restrict__ big, float* __restrict__ small,
                                           long long ldd, int rows, int cols, long long block,
                                           long long nblocks) {
  const long long groups = ldd / 4;
  const long long total = static_cast<long long>(rows) * groups;
  const bool vec = (reinterpret_cast<uintptr_t>(src) & 15u) == 0 && (lds & 3) == 0;
  for (long long g = block * blockDim.x + threadIdx.x; g < total; g += nblocks * blockDim.x) {
    const int r = static_cast<int>(g / groups);
    const int c0 = static_cast<int>(g % groups) * 4;
    const float* p = src + static_cast<long long>(r) * lds + c0;
    float x[4];
    if (vec && c0 + 4 <= cols) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(p));
      x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = (c0 + i < cols) ? __ldg(p + i) : 0.0f;
    }
    float b[4], s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) split_tf32(x[i], b[i], s[i]);
    const long long o = static_cast<long long>(r) * ldd + c0;
    *reinterpret_cast<float4*>(big + o) = make_float4(b[0], b[1], b[2], b[3]);
    *reinterpret_cast<float4*>(small + o) = make_float4(s[0], s[1], s[2], s[3]);
  }
}

// Transposing split of 32 x 32 tiles through shared memory (256 threads):
// src is rows x cols; dst rows are src columns (leading dimension ldd >= rows,
// % 4 == 0, zero padding in [rows, ldd)).  Thread t loads the 16 bytes at
// columns 4*(t % 8) of tile row t / 8 and stores the 16 bytes at columns
// 4*(t % 8) of tile row t / 8 of the transpose; tile[32][33] keeps the
// column reads of the store phase free of bank conflicts.  Element accesses
// when src or lds is not 16-byte aligned.
__device__ __forceinline__ void split_transpose(const float* __restrict__ src, long long lds,
                                                float* __restrict__ big, float* __restrict__ small,
                                                long long ldd, int rows, int cols, long long block,
                                                long long nblocks, float (*tile)[33]) {
  const int tiles_c = (cols + 31) / 32;
  const int tiles_r = static_cast<int>((ldd + 31) / 32);
  const long long ntiles = static_cast<long long>(tiles_r) * tiles_c;
  const bool vec = (reinterpret_cast<uintptr_t>(src) & 15u) == 0 && (lds & 3) == 0;
  const int tr = static_cast<int>(threadIdx.x) >> 3, tq = (static_cast<int>(threadIdx.x) & 7) * 4;
  for (long long t = block; t < ntiles; t += nblocks) {
    const int r0 = static_cast<int>(t / tiles_c) * 32, c0 = static_cast<int>(t % tiles_c) * 32;
    {
      const int rr = r0 + tr, cc = c0 + tq;
      const float* p = src + static_cast<long long>(rr) * lds + cc;
      float x[4];
      if (vec && rr < rows && cc + 4 <= cols) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(p));
        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = (rr < rows && cc + i < cols) ? __ldg(p + i) : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) tile[tr][tq + i] = x[i];
    }
    __syncthreads();
    {
      const int cc = c0 + tr, rr = r0 + tq;   // destination row cc, columns rr .. rr+3
      if (cc < cols && rr < ldd) {
        float b[4], sm[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) split_tf32(tile[tq + i][tr], b[i], sm[i]);
        const long long o = static_cast<long long>(cc) * ldd + rr;
        *reinterpret_cast<float4*>(big + o) = make_float4(b[0], b[1], b[2], b[3]);
        *reinterpret_cast<float4*>(small + o) = make_float4(sm[0], sm[1], sm[2], sm[3]);
      }
    }
    __syncthreads();
  }
}

// Both splits of a 3xTF32 product in one launch: blocks [0, grid_a) split A
// (M x K), the others split B^T (B is K x N).
__global__ void split_tf32_ab_kernel(const float* __restrict__ A, long long lda,
                                     float* __restrict__ Ab, float* __restrict__ As,
                                     const float* __restrict__ B, long long ldb,
                                     float* __restrict__ Bb, float* __restrict__ Bs, long long ld2,
                                     int M, int N, int K, int grid_a) {
  __shared__ float tile[32][33];
  if (static_cast<int>(blockIdx.x) < grid_a)
    split_rows(A, lda, Ab, As, ld2, M, K, blockIdx.x, grid_a);
  else
    split_transpose(B, ldb, Bb, Bs, ld2, K, N, blockIdx.x - grid_a, gridDim.x - grid_a, tile);
  // as for the realignment: the GEMM launched next may be scheduled
  griddep_launch_dependents();
}

// ---- fp32 operands as two scaled fp16 parts (the 3xFP16 SGEMM) ----------
// x * 2^e = h1 + h2 + r with h1 = half(x * 2^e) and h2 = half(x * 2^e - h1),
// both rounded to nearest: |r| <= 2^-22 |x * 2^e| (the same 11 + 11
// significand bits as the tf32 split).  e is a power-of-two exponent per row
// of A and per column of B within each K chunk of kF16x3ChunkK (the GEMM's
// accumulation chunk), chosen so that the largest magnitude of the row's
// (column's) chunk lands in [2^14, 2^15): no part overflows half, and the
// scaling and its undoing, chunk by chunk in the GEMM, are exact.  Chunks make
// every split local: one pass over each operand, no pass for maxima first.

// Exponent that takes the largest magnitude m into [2^14, 2^15); 0 when m is
// zero or not finite (the parts then carry the Inf or NaN).
__device__ __forceinline__ int f16x3_exponent(float m) {
  return (m > 0.0f && isfinite(m)) ? 14 - ilogbf(m) : 0;
}

// 2^e as two normal powers of two whose product is 2^e (e in [-113, 163]):
// x * f.x * f.y is then exact for every x the scaling is meant for.
__device__ __forceinline__ float2 f16x3_factors(int e) {
  const int e1 = max(-126, min(127, e));
  const int e2 = e - e1;   // 0 unless e > 127
  return make_float2(__int_as_float((e1 + 127) << 23), __int_as_float((e2 + 127) << 23));
}

__device__ __forceinline__ uint32_t f16x3_parts(float x, float2 f, uint32_t* lo) {
  const float y = (x * f.x) * f.y;
  const __half h1 = __float2half_rn(y);
  const __half h2 = __float2half_rn(y - __half2float(h1));
  *lo = __half_as_ushort(h2);
  return __half_as_ushort(h1);
}

// Four consecutive floats from a[k..k+3], zero past n (16-byte load when vec).
__device__ __forceinline__ float4 f16x3_load4(const float* a, int k, int n, bool vec) {
  if (vec && k + 4 <= n) return __ldcs(reinterpret_cast<const float4*>(a + k));
  float x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = (k + i < n) ? __ldcs(a + k + i) : 0.0f;
  return make_float4(x[0], x[1], x[2], x[3]);
}

// The two parts of four values with the factors f, as two 8-byte stores.
__device__ __forceinline__ void f16x3_put4(uint16_t* d1, uint16_t* d2, float4 v, float2 f) {
  uint32_t h[4], l[4];
  h[0] = f16x3_parts(v.x, f, &l[0]);
  h[1] = f16x3_parts(v.y, f, &l[1]);
  h[2] = f16x3_parts(v.z, f, &l[2]);
  h[3] = f16x3_parts(v.w, f, &l[3]);
  __stcs(reinterpret_cast<uint2*>(d1), make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16)));
  __stcs(reinterpret_cast<uint2*>(d2), make_uint2(l[0] | (l[1] << 16), l[2] | (l[3] << 16)));
}

__device__ __forceinline__ void f16x3_put4(uint16_t* d1, uint16_t* d2, float4 v, const float2 (&f)[4]) {
  uint32_t h[4], l[4];
  h[0] = f16x3_parts(v.x, f[0], &l[0]);
  h[1] = f16x3_parts(v.y, f[1], &l[1]);
  h[2] = f16x3_parts(v.z, f[2], &l[2]);
  h[3] = f16x3_parts(v.w, f[3], &l[3]);
  __stcs(reinterpret_cast<uint2*>(d1), make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16)));
  __stcs(reinterpret_cast<uint2*>(d2), make_uint2(l[0] | (l[1] << 16), l[2] | (l[3] << 16)));
}

// A, one warp per (row, chunk) item: the chunk's 256 values are two float4s
// per lane, held in registers between the maximum and the split; ea[row][c] =
// the exponent.
__device__ __forceinline__ void f16x3_split_a(const float* __restrict__ A, long long lda,
                                              uint16_t* __restrict__ A1, uint16_t* __restrict__ A2,
                                              long long ld2, int* __restrict__ ea, int M, int K,
                                              int kc, long long block, long long nblocks) {
  static_assert(kF16x3ChunkK == 256, "a chunk is two float4s per lane");
  const int lane = static_cast<int>(threadIdx.x & 31u);
  const long long warps = nblocks * (blockDim.x / 32);
  const bool vec = (reinterpret_cast<uintptr_t>(A) & 15u) == 0 && lda % 4 == 0;
  const long long items = static_cast<long long>(M) * kc;
  for (long long it = block * (blockDim.x / 32) + threadIdx.x / 32; it < items; it += warps) {
    const int r = static_cast<int>(it / kc), c = static_cast<int>(it % kc);
    const float* const a = A + r * lda;
    const int k0 = c * kF16x3ChunkK + 4 * lane, k1 = k0 + 128;
    const float4 v0 = f16x3_load4(a, k0, K, vec), v1 = f16x3_load4(a, k1, K, vec);
    float m = fmaxf(fmaxf(fmaxf(fabsf(v0.x), fabsf(v0.y)), fmaxf(fabsf(v0.z), fabsf(v0.w))),
                    fmaxf(fmaxf(fabsf(v1.x), fabsf(v1.y)), fmaxf(fabsf(v1.z), fabsf(v1.w))));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const int e = f16x3_exponent(m);
    const float2 f = f16x3_factors(e);
    if (lane == 0) ea[static_cast<long long>(r) * kc + c] = e;
    uint16_t* const d1 = A1 + r * ld2;
    uint16_t* const d2 = A2 + r * ld2;
    // groups of 4 elements (ld2 % 8 == 0; a group that crosses K gets zeros)
    if (k0 < K) f16x3_put4(d1 + k0, d2 + k0, v0, f);
    if (k1 < K) f16x3_put4(d1 + k1, d2 + k1, v1, f);
  }
}

// B, one block of kF16x3Threads threads per (chunk, 128 columns) item: warp w
// takes the chunk's rows kRowsPerWarp * w .. + kRowsPerWarp - 1 (all its loads
// in flight at once, held in registers), lane l columns 4l .. 4l + 3.  The
// column maxima go through shared memory, then each thread writes the parts
// of the values it holds; eb[c][col] = the exponent.  (With 256-thread blocks,
// 32 rows a warp and a second read of B the item was latency-bound.)
constexpr int kF16x3Threads = 1024;
constexpr int kF16x3Warps = kF16x3Threads / 32;
constexpr int kRowsPerWarp = kF16x3ChunkK / kF16x3Warps;
__device__ __forceinline__ void f16x3_split_b(const float* __restrict__ B, long long ldb,
                                              uint16_t* __restrict__ B1, uint16_t* __restrict__ B2,
                                              long long ld2, int* __restrict__ eb, long long ldeb,
                                              int K, int N, int kc, long long block,
                                              long long nblocks, float (&red)[kF16x3Warps][128],
                                              int (&es)[128]) {
  const int tid = static_cast<int>(threadIdx.x);
  const int lane = tid & 31, w = tid >> 5;
  const bool vec = (reinterpret_cast<uintptr_t>(B) & 15u) == 0 && ldb % 4 == 0;
  const int groups = (N + 127) / 128;
  const long long items = static_cast<long long>(kc) * groups;
  for (long long it = block; it < items; it += nblocks) {
    const int c = static_cast<int>(it / groups), g = static_cast<int>(it % groups);
    const int col = g * 128 + 4 * lane;
    const int r0 = c * kF16x3ChunkK + kRowsPerWarp * w;
    float4 v[kRowsPerWarp];
#pragma unroll
    for (int i = 0; i < kRowsPerWarp; ++i)
      v[i] = (r0 + i < K) ? f16x3_load4(B + static_cast<long long>(r0 + i) * ldb, col, N, vec)
                          : make_float4(0.f, 0.f, 0.f, 0.f);
    float m[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kRowsPerWarp; ++i) {
      m[0] = fmaxf(m[0], fabsf(v[i].x));
      m[1] = fmaxf(m[1], fabsf(v[i].y));
      m[2] = fmaxf(m[2], fabsf(v[i].z));
      m[3] = fmaxf(m[3], fabsf(v[i].w));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) red[w][4 * lane + j] = m[j];
    __syncthreads();
    if (tid < 128) {
      float mm = red[0][tid];
#pragma unroll
      for (int u = 1; u < kF16x3Warps; ++u) mm = fmaxf(mm, red[u][tid]);
      const int e = f16x3_exponent(mm);
      es[tid] = e;
      if (g * 128 + tid < N) eb[c * ldeb + g * 128 + tid] = e;
    }
    __syncthreads();
    if (col < N) {
      float2 f[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = f16x3_factors(es[4 * lane + j]);
#pragma unroll
      for (int i = 0; i < kRowsPerWarp; ++i) {   // the rows' values are still in registers
        const int k = r0 + i;
        if (k < K) f16x3_put4(B1 + k * ld2 + col, B2 + k * ld2 + col, v[i], f);
      }
    }
    __syncthreads();   // red and es are reused by the next item
  }
}

// One launch: blocks [0, grid_b) split B, the others A.
__global__ void __launch_bounds__(kF16x3Threads) f16x3_split_kernel(const float* __restrict__ A, long long lda,
                                   const float* __restrict__ B, long long ldb, const F16x3Parts p,
                                   int M, int N, int K, int grid_b) {
  __shared__ float red[kF16x3Warps][128];
  __shared__ int es[128];
  const int kc = (K + kF16x3ChunkK - 1) / kF16x3ChunkK;
  if (static_cast<int>(blockIdx.x) < grid_b)
    f16x3_split_b(B, ldb, p.B1, p.B2, p.ldb2, p.eb, p.ldeb, K, N, kc, blockIdx.x, grid_b, red, es);
  else
    f16x3_split_a(A, lda, p.A1, p.A2, p.lda2, p.ea, M, K, kc, blockIdx.x - grid_b,
                  gridDim.x - grid_b);
  // as for the realignment: the GEMM launched next may be scheduled
  griddep_launch_dependents();
}

// dst[i] = src[i] rounded to the nearest half (ties to even), eight elements
// per thread and step: two 16-byte loads and one 16-byte store when both
// pointers are 16-byte aligned (VEC), element accesses otherwise.
template <bool VEC>
__global__ void f32_to_f16_kernel(const float* __restrict__ src, uint16_t* __restrict__ dst,
                                  long long n) {
  const long long groups = (n + 7) / 8;
  for (long long g = blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x; g < groups;
       g += static_cast<long long>(gridDim.x) * blockDim.x) {
    const long long i = 8 * g;
    if (VEC && i + 8 <= n) {
      const float4 a = __ldcs(reinterpret_cast<const float4*>(src + i));
      const float4 b = __ldcs(reinterpret_cast<const float4*>(src + i) + 1);
      const __half2 h0 = __floats2half2_rn(a.x, a.y), h1 = __floats2half2_rn(a.z, a.w);
      const __half2 h2 = __floats2half2_rn(b.x, b.y), h3 = __floats2half2_rn(b.z, b.w);
      uint4 o;
      memcpy(&o.x, &h0, 4);
      memcpy(&o.y, &h1, 4);
      memcpy(&o.z, &h2, 4);
      memcpy(&o.w, &h3, 4);
      __stcs(reinterpret_cast<uint4*>(dst + i), o);
    } else {
      for (long long j = i; j < n && j < i + 8; ++j) dst[j] = __half_as_ushort(__float2half_rn(src[j]));
    }
  }
}

// One thread waits (bounded) on an mbarrier that nothing arrives on: the wait
// runs out after limit_ns, records GEMM_ERR_TIMEOUT in the status word and the
// kernel returns normally.  Used by the failure-detection test.
__global__ void wait_probe_kernel(unsigned long long limit_ns, DeviceStatus* st) {
  __shared__ __align__(8) uint64_t bar;
  const uint32_t b = smem_addr(&bar);
  mbar_init(b, 1u);
  fence_barrier_init();
  wait_parity(b, 0u, limit_ns, st, 99);
}

}  // namespace

cudaError_t launch_wait_probe(unsigned long long limit_ns, DeviceStatus* status,
                              cudaStream_t stream) {
  wait_probe_kernel<<<1, 1, 0, stream>>>(limit_ns, status);
  return counted_launch(cudaGetLastError());
}

cudaError_t launch_f32_to_f16(const float* src, uint16_t* dst, long long n, int grid,
                              cudaStream_t stream) {
  const bool vec = ((reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst)) & 15u) == 0;
  if (vec)
    f32_to_f16_kernel<true><<<grid, 256, 0, stream>>>(src, dst, n);
  else
    f32_to_f16_kernel<false><<<grid, 256, 0, stream>>>(src, dst, n);
  return counted_launch(cudaGetLastError());
}

cudaError_t launch_split_tf32_ab(const float* A, long long lda, float* Ab, float* As,
                                 const float* B, long long ldb, float* Bb, float* Bs, long long ld2,
                                 int M, int N, int K, int grid_a, int grid_b, cudaStream_t stream) {
  split_tf32_ab_kernel<<<grid_a + grid_b, 256, 0, stream>>>(A, lda, Ab, As, B, ldb, Bb, Bs, ld2, M,
                                                            N, K, grid_a);
  return counted_launch(cudaGetLastError());
}


cudaError_t launch_f16x3_split(const float* A, long long lda, const float* B, long long ldb,
                               const F16x3Parts& p, int M, int N, int K, int grid_a, int grid_b,
                               cudaStream_t stream) {
  f16x3_split_kernel<<<grid_a + grid_b, kF16x3Threads, 0, stream>>>(A, lda, B, ldb, p, M, N, K,
                                                                      grid_b);
  return counted_launch(cudaGetLastError());
}

cudaError_t launch_realign_f16(const RealignBatch& batch, cudaStream_t stream) {
  if (batch.n < 1 || batch.n > kRealignJobs) return cudaErrorInvalidValue;
  const unsigned grid = static_cast<unsigned>(batch.end[batch.n - 1]);
  if (batch.early) return counted_launch(launch_early(realign_f16_kernel, grid, 256, 0, stream, batch));
  realign_f16_kernel<<<grid, 256, 0, stream>>>(batch);
  return counted_launch(cudaGetLastError());
}

cudaError_t launch_unalign_f16(const RealignBatch& batch, cudaStream_t stream) {
  if (batch.n < 1 || batch.n > kRealignJobs) return cudaErrorInvalidValue;
  return counted_launch(launch_early(unalign_f16_kernel, static_cast<unsigned>(batch.end[batch.n - 1]),
                                     256, 0, stream, batch));
}

cudaError_t launch_splitk_reduce_f16(const float* ws, long long ws_ld, int splits, uint16_t* C,
                                     long long ldc, int M, int N, float alpha, float beta,
                                     int grid, cudaStream_t stream) {
  splitk_reduce_f16_kernel<<<grid, 256, 0, stream>>>(ws, ws_ld, splits, C, ldc, M, N, alpha, beta);
  return counted_launch(cudaGetLastError());
}

cudaError_t launch_scale_f16(uint16_t* C, long long ldc, int M, int N, float beta, int grid,
                             cudaStream_t stream) {
  scale_f16_kernel<<<grid, 256, 0, stream>>>(C, ldc, M, N, beta);
  return counted_launch(cudaGetLastError());
}

cudaError_t launch_scale_f32(float* C, long long ldc, int M, int N, float beta, int grid,
                             cudaStream_t stream) {
  scale_f32_kernel<<<grid, 256, 0, stream>>>(C, ldc, M, N, beta);
  return counted_launch(cudaGetLastError());
}

}  // namespace gb300
