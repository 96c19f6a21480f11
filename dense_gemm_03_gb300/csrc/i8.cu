// i8.cu -- products in 8-bit integers with a scale for each token and channel, and the
// rounding of tokens to 8 bits: argument checks, path choice and the kernels that
// turn rows of halves into rows of integers and back.
//
//   product    S = X W, C := sx[i] sw[n] S + beta C, or gated.  Products are exact in fp32, and S is
//              while its partial sums stay below 2^24 (whatever the values up to K = 1024);
//              past that it is rounded, the tensor core truncating, as a product of halves is
//   tokens     a = max_k |X[i,k]|, scale[i] = a / 127, Q[i,k] = round(127 X[i,k] / a)
//
// Few rows or few tiles: i8_stream.cu (bytes to halves on their way to the tensor
// cores).  Else both operands become halves in scratch, read back
// from L2 by the pair kernel (gemm_f16_tc_kernel.cuh), whose epilogue scales.
#include <cuda_fp16.h>

#include "gemm.h"
#include "i8_convert.cuh"
#include "lora.h"
#include "operands.h"
#include "ptx_i8.cuh"
#include "stream.h"

namespace gb300 {
namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------- integers to halves
// dst[r][c] = src[r][c] for c < cols, 0 for cols <= c < width (a multiple of 16); one
// thread 16 elements, dst rows on the 16-byte grid.
struct SpreadJob {
  const int8_t* src;
  long long lds;
  void* dst;
  long long ldd;
  int rows, cols, width;
};
constexpr int kSpreadJobs = 3;
struct SpreadBatch {
  SpreadJob job[kSpreadJobs];
  int end[kSpreadJobs];   // blocks [end[i-1], end[i]) do job i
  int n;
};

// 16 bytes at any address, of which `n` belong to the row.
__device__ __forceinline__ uint4 load16(const int8_t* p, int n) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  if (n >= 16 && (a & 15u) == 0) return __ldg(reinterpret_cast<const uint4*>(p));
  uint32_t w[4] = {0u, 0u, 0u, 0u};
  if (n >= 16) {
    // the one or two aligned blocks that hold the piece (each holds bytes of it)
    const uint32_t m = static_cast<uint32_t>(a & 15u);
    const uint4* const blk = reinterpret_cast<const uint4*>(a - m);
    const uint4 lo = __ldg(blk), hi = __ldg(blk + 1);
    const uint32_t v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    const uint32_t sh = (m & 3u) * 8u;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (static_cast<int>(m >> 2) == q)
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(v[q + i], v[q + i + 1 < 8 ? q + i + 1 : 7], sh);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) w[i >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(__ldg(p + i))) << (8 * (i & 3));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// HALVES: as halves (every 8-bit integer is one), else as bytes on the 16-byte grid.
template <bool HALVES>
__global__ void __launch_bounds__(kThreads) spread_i8_kernel(const SpreadBatch b) {
  griddep_launch_dependents();
  griddep_wait();
  int i = 0;
  while (i + 1 < b.n && static_cast<int>(blockIdx.x) >= b.end[i]) ++i;
  const int first = i ? b.end[i - 1] : 0;
  const SpreadJob& j = b.job[i];
  const int groups = j.width / 16;
  const long long total = static_cast<long long>(j.rows) * groups;
  for (long long g = (blockIdx.x - first) * static_cast<long long>(kThreads) + threadIdx.x; g < total;
       g += static_cast<long long>(b.end[i] - first) * kThreads) {
    const int r = static_cast<int>(g / groups), c = static_cast<int>(g - static_cast<long long>(r) * groups) * 16;
    const uint4 q = load16(j.src + r * j.lds + c, j.cols - c);
    const long long at = r * j.ldd + c;
    if constexpr (!HALVES) {
      *reinterpret_cast<uint4*>(static_cast<int8_t*>(j.dst) + at) = q;
    } else {
      uint4* const dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(j.dst) + at);
      i8_halves16(q, dst[0], dst[1]);
    }
  }
}

int spread(SpreadBatch& b, bool halves, int sms, cudaStream_t stream) {
  int blocks = 0;
  for (int i = 0; i < b.n; ++i) {
    const long long want = (1ll * b.job[i].rows * (b.job[i].width / 16) + kThreads - 1) / kThreads;
    blocks += static_cast<int>(std::max(1ll, std::min<long long>(want, 16ll * sms)));
    b.end[i] = blocks;
  }
  return counted_launch(launch_early(halves ? spread_i8_kernel<true> : spread_i8_kernel<false>,
                                     blocks, kThreads, 0, stream, b)) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

// ------------------------------------------------------------ tokens to bytes
// T threads a row, V groups of eight elements a thread kept in registers between the
// two passes over them (V == 0: a row too long for that, read twice).  Groups lie on
// Q's 8-byte grid, so that stores are whole; a row's first and last may be ragged.
//
// The maximum is taken over the bits of |x|, which order like the values, infinities
// above them and NaNs above those.  127 x / a is x times 127 / a, the latter rounded up,
// and rounds to an integer as 1.5 2^23 is added (one rounding, of the exact product).
// That is exact.  With significands X and A below 2^11, 127 x / a - (k + 1/2) is zero or at
// least 2^-19 of the quotient, and the product is off by at most 2^-23 of it.  A tie, 254 x
// = (2k + 1) a, has 127 among the factors of 2k + 1 or of A.  2k + 1 = 127 is x = a / 2,
// whose product is 63.5 or a little more and rounds to 64, the even one; rows whose A is a
// multiple of 127 divide instead (127 x is exact, and so is a tie's quotient).
struct RowScale {
  float a, inv;         // the maximum, 127 / a rounded up (0: the row's integers are zeros)
  bool finite, divide;
};

__device__ __forceinline__ RowScale row_scale(uint32_t bits) {   // of the maximum, as a half
  RowScale s;
  s.a = lora_h2f(static_cast<uint16_t>(bits));
  s.finite = bits < 0x7C00u;
  s.inv = bits != 0u && s.finite ? __fdiv_ru(127.0f, s.a) : 0.0f;
  const uint32_t significand = (bits & 0x3FFu) | (bits >= 0x400u ? 0x400u : 0u);
  s.divide = s.finite && bits != 0u && significand % 127u == 0u;
  return s;
}

// The larger of each half's magnitude bits.
__device__ __forceinline__ uint32_t max_bits(uint32_t m, uint4 v) {
  constexpr uint32_t kAbs = 0x7FFF7FFFu;
  return __vmaxu2(m, __vmaxu2(__vmaxu2(v.x & kAbs, v.y & kAbs), __vmaxu2(v.z & kAbs, v.w & kAbs)));
}

// Eight halves as integers, one to a byte.
__device__ __forceinline__ uint2 round_row8(const RowScale& s, uint4 v) {
  constexpr float kMagic = 12582912.0f;   // 1.5 2^23: the integer is in the low bits
  if (!s.finite) v = make_uint4(0u, 0u, 0u, 0u);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 h = lora_h2f2(w[i]);
    b[2 * i] = __float_as_uint(fmaf(h.x, s.inv, kMagic));
    b[2 * i + 1] = __float_as_uint(fmaf(h.y, s.inv, kMagic));
  }
  if (s.divide)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 h = lora_h2f2(w[i]);
      b[2 * i] = __float_as_uint(__fadd_rn(__fdiv_rn(127.0f * h.x, s.a), kMagic));
      b[2 * i + 1] = __float_as_uint(__fadd_rn(__fdiv_rn(127.0f * h.y, s.a), kMagic));
    }
  return make_uint2(
      __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410),
      __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410));
}

template <int T, int V>
__global__ void __launch_bounds__(T < 256 ? 256 : T)
    to_i8_kernel(const uint16_t* __restrict__ X, int8_t* __restrict__ Q, float* __restrict__ scales,
                 int M, int K, long long ldx, long long ldq) {
  constexpr int kRowsPerBlock = T < 256 ? 256 / T : 1;
  __shared__ uint32_t top[32];
  griddep_launch_dependents();
  griddep_wait();
  const int t = static_cast<int>(threadIdx.x) % T;
  const int row = blockIdx.x * kRowsPerBlock + static_cast<int>(threadIdx.x) / T;
  const bool there = row < M;   // (uniform over a warp)
  const uint16_t* const x = X + (there ? row * ldx : 0);
  int8_t* const q = Q + (there ? row * ldq : 0);
  const int md = static_cast<int>(reinterpret_cast<uintptr_t>(q) & 7u);
  const int groups = there ? (K + md + 7) / 8 : 0;
  auto load = [&](int j) {
    const int e0 = 8 * j - md;
    if (e0 >= 0 && e0 + 8 <= K) {
      const uintptr_t a = reinterpret_cast<uintptr_t>(x + e0);
      const uint32_t m = static_cast<uint32_t>(a & 15u);
      const uint4* const blk = reinterpret_cast<const uint4*>(a - m);
      const uint4 lo = __ldg(blk);
      if (m == 0) return lo;
      const uint4 hi = __ldg(blk + 1);   // (holds elements of the group)
      const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
      const uint32_t sh = (m & 3u) * 8u;
      uint32_t o[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int s = 0; s < 4; ++s)
        if (static_cast<int>(m >> 2) == s)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = __funnelshift_r(w[s + i], w[s + i + 1 < 8 ? s + i + 1 : 7], sh);
      return make_uint4(o[0], o[1], o[2], o[3]);
    }
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = e0 + i >= 0 && e0 + i < K ? __ldg(x + e0 + i) : 0u;
    return make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
  };
  uint32_t m2 = 0u;
  auto look = [&](uint4 v) { m2 = max_bits(m2, v); };
  uint4 kept[V > 0 ? V : 1];
  if constexpr (V > 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) kept[i] = t + T * i < groups ? load(t + T * i) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < V; ++i) look(kept[i]);
  } else {
    for (int j = t; j < groups; j += T) look(load(j));
  }
  uint32_t bits = max(m2 & 0xFFFFu, m2 >> 16);
  bits = __reduce_max_sync(0xffffffffu, bits);
  if constexpr (T > 32) {
    const int warp = static_cast<int>(threadIdx.x) / 32;
    if ((threadIdx.x & 31) == 0) top[warp] = bits;
    __syncthreads();
    bits = top[0];
#pragma unroll
    for (int i = 1; i < T / 32; ++i) bits = max(bits, top[i]);
  }
  if (!there) return;
  const RowScale scale = row_scale(bits);
  if (t == 0) scales[row] = __fdiv_rn(scale.a, 127.0f);
  auto put = [&](int j, uint4 v) {
    const uint2 b = round_row8(scale, v);
    const int e0 = 8 * j - md;
    if (e0 >= 0 && e0 + 8 <= K) {
      *reinterpret_cast<uint2*>(q + e0) = b;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e0 + i >= 0 && e0 + i < K)
          q[e0 + i] = static_cast<int8_t>(((i < 4 ? b.x : b.y) >> (8 * (i & 3))) & 0xFFu);
    }
  };
  if constexpr (V > 0) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (t + T * i < groups) put(t + T * i, kept[i]);
  } else {
    for (int j = t; j < groups; j += T) put(j, load(j));
  }
}

// The same for many rows on the 16-byte grid: persistent blocks, each with a ring of
// rows in shared memory that bulk copies fill, so that loads are always in flight
// (single rows a block: 45 us for 8192 x 8192; a copy of as many bytes takes 35).  T
// threads a row, V pieces of 16 elements each; a group of T threads has every
// (kRingThreads / T)-th stage to itself and refills it as soon as its threads hold the row.
constexpr int kRingThreads = 512;
constexpr int kRingBytes = 196608;
constexpr int kRingStages = 48;

template <int T, int V>
__global__ void __launch_bounds__(kRingThreads, 1)
    to_i8_ring_kernel(const uint16_t* __restrict__ X, int8_t* __restrict__ Q,
                      float* __restrict__ scales, int M, int K, long long ldx, long long ldq,
                      int stages, unsigned long long limit, DeviceStatus* st) {
  constexpr int kGroups = kRingThreads / T;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(8) unsigned long long bars[kRingStages];
  __shared__ uint32_t top[2][kRingThreads / 32];
  const int group = static_cast<int>(threadIdx.x) / T, t = static_cast<int>(threadIdx.x) % T;
  const int warp = static_cast<int>(threadIdx.x) / 32;
  const uint32_t bytes = static_cast<uint32_t>(2 * K);
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(smem_addr(&bars[s]), 1u);
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  __syncthreads();
  griddep_launch_dependents();
  griddep_wait();
  // row number i of this block, in stage i % stages
  auto row_of = [&](long long i) { return blockIdx.x + i * gridDim.x; };
  auto fetch = [&](long long i, int s) {
    const uint32_t bar = smem_addr(&bars[s]);
    mbar_arrive_expect_tx(bar, bytes);
    bulk_load(smem_addr(ring + static_cast<size_t>(s) * bytes), X + row_of(i) * ldx, bytes, bar);
  };
  if (t == 0)
    for (int s = group; s < stages; s += kGroups)
      if (row_of(s) < M) fetch(s, s);
  bool ok = true;
  int s = group, turn = 0;
  uint32_t phase = 0;
  for (long long i = group; ok && row_of(i) < M; i += kGroups, turn ^= 1) {
    const long long row = row_of(i);
    ok = wait_parity(smem_addr(&bars[s]), phase, limit, st, 80);
    const uint4* const src = reinterpret_cast<const uint4*>(ring + static_cast<size_t>(s) * bytes);
    uint4 v[V][2];
    uint32_t m2 = 0u;
#pragma unroll
    for (int u = 0; u < V; ++u) {
      const int e = t + T * u;   // piece of 16
#pragma unroll
      for (int h = 0; h < 2; ++h)
        v[u][h] = 16 * e < K ? src[2 * e + h] : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int u = 0; u < V; ++u) m2 = max_bits(max_bits(m2, v[u][0]), v[u][1]);
    constexpr uint32_t kGaveUp = 0xFFFFFFFFu;   // one thread's wait did: the whole group's
    uint32_t bits = __reduce_max_sync(0xffffffffu, ok ? max(m2 & 0xFFFFu, m2 >> 16) : kGaveUp);
    if constexpr (T > 32) {
      if ((threadIdx.x & 31) == 0) top[turn][warp] = bits;
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(T) : "memory");
#pragma unroll
      for (int w = 0; w < T / 32; ++w) bits = max(bits, top[turn][group * (T / 32) + w]);
    }
    ok = bits != kGaveUp;
    if (!ok) break;
    // every thread of the group holds its part of the row
    if (t == 0 && row_of(i + stages) < M) fetch(i + stages, s);
    const RowScale scale = row_scale(bits);
    if (t == 0) scales[row] = __fdiv_rn(scale.a, 127.0f);
#pragma unroll
    for (int u = 0; u < V; ++u) {
      const int e = t + T * u;
      if (16 * e < K) {
        const uint2 lo = round_row8(scale, v[u][0]), hi = round_row8(scale, v[u][1]);
        __stcs(reinterpret_cast<uint4*>(Q + row * ldq) + e, make_uint4(lo.x, lo.y, hi.x, hi.y));
      }
    }
    s += kGroups;
    if (s >= stages) {
      s -= stages;
      phase ^= 1u;
    }
  }
  // a wait that gave up leaves copies in flight
  if (!ok && t == 0)
    for (int r = group; r < stages; r += kGroups) {
      settle_wait(smem_addr(&bars[r]), 0u, st, 81);
      settle_wait(smem_addr(&bars[r]), 1u, st, 81);
    }
}

template <int T, int V>
int launch_ring(const uint16_t* X, int8_t* Q, float* scales, int M, int K, int ldx, int ldq,
                const LoraDevice& d, cudaStream_t stream) {
  constexpr int kGroups = kRingThreads / T;
  static bool configured[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return GEMM_ERR_CUDA;
  if (dev < 64 && !configured[dev]) {
    if (cudaFuncSetAttribute(to_i8_ring_kernel<T, V>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kRingBytes) != cudaSuccess)
      return GEMM_ERR_CUDA;
    configured[dev] = true;
  }
  const int stages = std::min(kRingStages, kRingBytes / (2 * K)) / kGroups * kGroups;
  return counted_launch(launch_early(to_i8_ring_kernel<T, V>, d.sms, kRingThreads,
                                     static_cast<size_t>(stages) * 2 * K, stream, X, Q, scales, M, K,
                                     static_cast<long long>(ldx), static_cast<long long>(ldq), stages,
                                     d.wait_limit_ns, d.status)) == cudaSuccess
             ? GEMM_OK
             : GEMM_ERR_CUDA;
}

__global__ void __launch_bounds__(kThreads) zero_floats_kernel(float* p, int n) {
  for (int i = blockIdx.x * kThreads + threadIdx.x; i < n; i += gridDim.x * kThreads) p[i] = 0.0f;
}

int device(LoraDevice* d) { return query_device(&d->sms, &d->status, &d->wait_limit_ns); }

struct I8Args {
  const int8_t *X, *W;
  const float *sx, *sw;
  uint16_t* C;
  int M, N, K, act, ldx, ldw, ldc;
  float beta;
  bool gated() const { return act != GEMM_ACT_NONE; }
  int cols() const { return gated() ? 2 * N : N; }
};

bool on_grid(const int8_t* p, int ld) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 16 == 0;
}

// Whether to convert W on its way (streamed), once for each block of 128 rows, or once and
// for all into scratch (tiled).  Estimates in us, from GB300: a 128-deep step of 128 rows
// and columns takes 0.6 where one wave of CTAs holds all tiles, else 0.85 of an SM; the tiled
// form makes, writes and reads back three bytes for each of W at 4.5 TB/s, then runs
// waves of tiles at 0.3 a k-block.  Measured, streamed against tiled: 4096 x 2*8192 with 384
// rows 75, 85, with 512 99, 85; 4096 x 4096 with 512 rows 27, 36, with 768 44, 39.
bool stream_suits(const I8Args& p, int sms) {
  if (p.M <= 128) return true;
  const double steps = (p.K + 127) / 128;
  const double units = 1.0 * ((p.M + 127) / 128) * ((p.cols() + 127) / 128);
  const double stream = 7 + steps * (units <= sms ? 0.6 : 0.85 * units / sms);
  const long long tiles = 1ll * ((p.M + 255) / 256) * ((p.cols() + 255) / 256);
  const long long waves = (2 * tiles + sms - 1) / sms;
  return stream < 0.85 * (17 + 3e-6 / 4.5 * p.K * p.cols() + 0.6 * waves * steps);
}

int streamed(const I8Args& p, const GateArgs& g, const LoraDevice& d, cudaStream_t stream) {
  NarrowStream r{p.X, p.W, p.ldx, p.ldw, p.K, false, false};
  StreamSum s{};
  s.C = p.C;
  s.ldc = p.ldc;
  s.M = p.M;
  s.N = p.N;
  s.alpha = 1.0f;
  s.beta = p.beta;
  s.gate = p.gated();
  s.scaled = true;
  s.g = g;
  const bool cluster = i8_cluster_suits(s, p.K, d);
  if (!cluster) s.parts = i8_parts(r, p.M, p.cols(), d);
  const bool copy_x = !on_grid(p.X, p.ldx), copy_w = !on_grid(p.W, p.ldw);
  const int kx = (p.K + 15) / 16 * 16, kw = (p.cols() + 15) / 16 * 16;
  const size_t x_bytes = copy_x ? lora_round256(static_cast<size_t>(p.M) * kx) : 0;
  const size_t w_bytes = copy_w ? lora_round256(static_cast<size_t>(p.K) * kw) : 0;
  void* buf = nullptr;
  if (x_bytes + w_bytes + s.parts.bytes)
    if (int rc = routed_scratch(stream, x_bytes + w_bytes + s.parts.bytes, &buf)) return rc;
  uint8_t* at = static_cast<uint8_t*>(buf);
  SpreadBatch b{};
  if (copy_x) {
    b.job[b.n++] = SpreadJob{p.X, p.ldx, at, kx, p.M, p.K, kx};
    r.X = at;
    r.ldx = kx;
  }
  at += x_bytes;
  if (copy_w) {
    b.job[b.n++] = SpreadJob{p.W, p.ldw, at, kw, p.K, p.cols(), kw};
    r.W = at;
    r.ldw = kw;
  }
  at += w_bytes;
  if (b.n)
    if (int rc = spread(b, false, d.sms, stream)) return rc;
  if (cluster) {
    if (int rc = i8_cluster(r, s, d, stream)) return rc;
  } else {
    s.parts.part = reinterpret_cast<float*>(at);
    if (int rc = i8_partial(r, p.M, p.cols(), s.parts, d, stream)) return rc;
    if (int rc = stream_sum(s, d, stream)) return rc;
  }
  set_last_path(b.n ? "i8.stream.realigned" : "i8.stream");
  return GEMM_OK;
}

int tiled(const I8Args& p, GateArgs g, const LoraDevice& d, cudaStream_t stream) {
  // the gate's columns and those it gates apart, each from a 16-byte boundary
  const bool apart = p.gated() && p.N % 8 != 0;
  const int kx = (p.K + 15) / 16 * 16, n16 = (p.N + 15) / 16 * 16;
  const int kw = apart ? 2 * n16 : (p.cols() + 15) / 16 * 16;
  const size_t x_bytes = lora_round256(2 * static_cast<size_t>(p.M) * kx);
  const size_t w_bytes = lora_round256(2 * static_cast<size_t>(p.K) * kw);
  void* buf = nullptr;
  if (int rc = routed_scratch(stream, x_bytes + w_bytes, &buf)) return rc;
  uint16_t* const x = static_cast<uint16_t*>(buf);
  uint16_t* const w = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(buf) + x_bytes);
  SpreadBatch b{};
  b.job[b.n++] = SpreadJob{p.X, p.ldx, x, kx, p.M, p.K, kx};
  if (apart) {
    b.job[b.n++] = SpreadJob{p.W, p.ldw, w, kw, p.K, p.N, n16};
    b.job[b.n++] = SpreadJob{p.W + p.N, p.ldw, w + n16, kw, p.K, p.N, n16};
  } else {
    b.job[b.n++] = SpreadJob{p.W, p.ldw, w, kw, p.K, p.cols(), kw};
  }
  if (int rc = spread(b, true, d.sms, stream)) return rc;
  PairCall q{};
  q.A = x;
  q.B = w;
  q.C = p.C;
  q.M = p.M;
  q.N = p.N;
  q.K = p.K;
  q.lda = kx;
  q.ldb = kw;
  q.ldc = p.ldc;
  q.alpha = 1.0f;
  q.beta = p.beta;
  q.gate = p.gated();
  q.scaled = true;
  q.g = g;
  q.g.up = apart ? n16 : p.N;
  return gemm_f16_pair(q, stream);
}

}  // namespace
}  // namespace gb300

using namespace gb300;

extern "C" {

int gemm_i8(const int8_t* X, const int8_t* W, uint16_t* C, const float* sx, const float* sw, int M,
            int N, int K, int act, int ldx, int ldw, int ldc, float beta, cudaStream_t stream) {
  if (M < 0 || N < 0 || K < 0) return GEMM_ERR_DIM;
  const bool gated = act != GEMM_ACT_NONE;
  if (act < GEMM_ACT_NONE || act > GEMM_ACT_RELU ||
      (gated && (beta != 0.0f || N > GEMM_GLU_MAX_N)) || std::max({M, N, K}) > kMaxDim)
    return GEMM_ERR_ARG;
  if (M == 0 || N == 0) {
    set_last_path("noop");
    return GEMM_OK;
  }
  if (ldc < N || (K > 0 && (ldx < K || ldw < (gated ? 2 * N : N)))) return GEMM_ERR_LD;
  if (!C || (K > 0 && (!X || !W))) return GEMM_ERR_NULL;
  if (misaligned({C}, 2) || misaligned({sx, sw}, 4)) return GEMM_ERR_ARG;
  LoraDevice d{};
  if (int rc = device(&d)) return rc;
  std::unique_lock<std::recursive_mutex> call;
  if (int rc = lock_stream(stream, &call)) return rc;
  if (K == 0) {
    set_last_path("i8.scale");
    return launch_scale_f16(C, ldc, M, N, beta, 8 * d.sms, stream) == cudaSuccess ? GEMM_OK
                                                                                 : GEMM_ERR_CUDA;
  }
  const I8Args p{X, W, sx, sw, C, M, N, K, act, ldx, ldw, ldc, beta};
  GateArgs g{};
  g.act = act;
  g.up = N;
  g.sx = sx;
  g.sw = sw;
  return stream_suits(p, d.sms) ? streamed(p, g, d, stream) : tiled(p, g, d, stream);
}

int gemm_f16_to_i8(const uint16_t* X, int8_t* Q, float* scales, int M, int K, int ldx, int ldq,
                   cudaStream_t stream) {
  if (M < 0 || K < 0) return GEMM_ERR_DIM;
  if (std::max(M, K) > kMaxDim) return GEMM_ERR_ARG;
  if (M == 0) {
    set_last_path("noop");
    return GEMM_OK;
  }
  if (K > 0 && (ldx < K || ldq < K)) return GEMM_ERR_LD;
  if (!scales || (K > 0 && (!X || !Q))) return GEMM_ERR_NULL;
  if (misaligned({X}, 2) || misaligned({scales}, 4)) return GEMM_ERR_ARG;
  LoraDevice d{};
  if (int rc = device(&d)) return rc;
  if (K == 0) {
    set_last_path("to_i8.blank");
    zero_floats_kernel<<<d.sms, kThreads, 0, stream>>>(scales, M);
    return counted_launch(cudaGetLastError()) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
  }
  set_last_path("to_i8");
  // rings from 12 million elements on: 4096 x 4096 12.4 us (14.2 by single rows), 4096 x
  // 2048 6.8 (7.3), but 2048 x 4096 7.1 (6.1) and 8192 x 1024 6.9 (6.3)
  if (K % 16 == 0 && ldx % 8 == 0 && ldq % 16 == 0 && !misaligned({X, Q}, 16) && K <= 16384 &&
      1ll * M * K >= 12ll << 20) {
    set_last_path("to_i8.ring");
    if (K <= 512) return launch_ring<32, 1>(X, Q, scales, M, K, ldx, ldq, d, stream);
    if (K <= 1024) return launch_ring<32, 2>(X, Q, scales, M, K, ldx, ldq, d, stream);
    if (K <= 2048) return launch_ring<32, 4>(X, Q, scales, M, K, ldx, ldq, d, stream);
    if (K <= 4096) return launch_ring<128, 2>(X, Q, scales, M, K, ldx, ldq, d, stream);
    if (K <= 8192) return launch_ring<128, 4>(X, Q, scales, M, K, ldx, ldq, d, stream);
    return launch_ring<256, 4>(X, Q, scales, M, K, ldx, ldq, d, stream);
  }
  // groups of a row: at most, when Q's rows leave its 8-byte grid
  const bool grid8 = (reinterpret_cast<uintptr_t>(Q) & 7u) == 0 && ldq % 8 == 0;
  const int groups = grid8 ? (K - 1) / 8 + 1 : K / 8 + 2;
  cudaError_t e = cudaSuccess;
  auto launch = [&](auto kernel, int threads, int rows) {
    e = launch_early(kernel, (M - 1) / rows + 1, threads, 0, stream, X, Q, scales, M, K,
                     static_cast<long long>(ldx), static_cast<long long>(ldq));
  };
  if (groups <= 32)
    launch(to_i8_kernel<32, 1>, 256, 8);
  else if (groups <= 64)
    launch(to_i8_kernel<32, 2>, 256, 8);
  else if (groups <= 128)
    launch(to_i8_kernel<32, 4>, 256, 8);
  else if (groups <= 256)
    launch(to_i8_kernel<256, 1>, 256, 1);
  else if (groups <= 512)
    launch(to_i8_kernel<256, 2>, 256, 1);
  else if (groups <= 1024)
    launch(to_i8_kernel<256, 4>, 256, 1);
  else if (groups <= 4096)
    launch(to_i8_kernel<1024, 4>, 1024, 1);
  else
    launch(to_i8_kernel<1024, 0>, 1024, 1);
  return counted_launch(e) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

}  // extern "C"
