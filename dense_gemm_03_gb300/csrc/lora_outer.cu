// lora_outer.cu -- the adapters' gradients, sums over the rows of each adapter:
//
//   dA[a] = alpha sum X_i^T U_i + beta dA[a],  dB[a] = alpha sum V_i^T dC_i + beta dB[a]
//
// lora_outer_kernel: one item is (512 rows, an adapter that occurs in them, 256
// columns of X or of dC, 32 ranks).  X (dC) is the M operand, as it lies in
// memory (MN-major, 64 rows a k-block); the N operand is the rows' U (V) in two
// halves, hi in columns 0 .. 31 and lo in 32 .. 63, so one product gives both
// parts.  What binds is reading X and dC once per adapter in the rows (once in
// all, when an adapter's rows lie together); the rest is small.  64-row blocks
// without the adapter are skipped.  Items write fp32 partial sums, which
// lora_outer_sum_kernel adds up in row order; up to 512 rows in all (one range)
// they write the gradients themselves (256 x 1024 x 1024: 23.4 -> 22.0 us).
//
// U and V come scaled by a power of two for each adapter of 128 rows
// (lora_shrink.cu); 64 rows are what is summed in TMEM (the tensor cores
// truncate, see there), and the scale is taken back as those sums are added up in
// registers.
//
// Rows of other adapters in a block have zeros for U (V), and their part of X
// (dC) is overwritten by zeros in shared memory, so that an Inf or NaN there
// stays with its own adapter.
#include "lora.h"

namespace gb300 {
namespace {

constexpr int kRange = 512;                  // rows of an item
constexpr int kLoaders = 4;
constexpr int kEpi = 8;                      // epilogue warps: four per accumulator
constexpr int kThreads = 32 * (2 + kLoaders + kEpi);
constexpr int kStages = 5;
constexpr int kXBytes = 4 * 64 * 128;        // 64 rows x 256 columns
constexpr int kVBytes = 64 * 128;            // 64 rows x (32 hi, 32 lo)
constexpr int kStageBytes = kXBytes + kVBytes;
constexpr int kTmemCols = 256;               // two buffers of two 64-column accumulators
constexpr int kMaxMasks = kLoraMaxAdapters;  // ranges x adapters of a launch
constexpr int kGroupMasks = 32;              // masks per entry of the prefix
constexpr int kBars = 3 * kStages + 5;
constexpr int kScales = 16;                  // blocks' scales on their way to the epilogue
// (a loader writes one before it waits for the block's stage: four blocks on from
// one whose stage was free, while the epilogue has two left)
static_assert(kScales >= kLoaders + kStages + 2, "places of scales still to be read");
constexpr int kSmem = 1024 + kStages * kStageBytes + 8 * kBars + 8 + 4 * kScales;
static_assert(kSmem + 16 + kMaxMasks + kMaxMasks / 8 + 64 <= 232448, "shared memory budget");

struct Args {
  const float *unscale_u, *unscale_v;   // by row
  int cols_x, cols_g, tiles_x, tiles_g;   // of X and dC, 256-column tiles (0: not wanted)
  const int* ids;
  int M, R, adapters, chunks, ranges, row0;
  float* part;             // [present][tile columns and ranks as in dA, then as in dB]
  long long part_stride, part_b;
  int* table;              // [range][adapter]: place among the present ones, or -1
  // one range (direct): the gradients themselves
  float *dA, *dB;
  float alpha, beta;
  int direct;
  unsigned long long wait_limit_ns;
  DeviceStatus* status;
};

struct Item {
  int present, range, a, mask, src, tile, chunk;
};

__global__ void __launch_bounds__(kThreads, 1)
    lora_outer_kernel(const __grid_constant__ CUtensorMap tmX,
                      const __grid_constant__ CUtensorMap tmG,
                      const __grid_constant__ CUtensorMap tmU,
                      const __grid_constant__ CUtensorMap tmV, const Args p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const base_ptr = smem_raw + (base - raw);
  const uint32_t bars = base + kStages * kStageBytes;
  auto full_bar = [&](int s) { return bars + 8u * s; };
  auto tok_bar = [&](int s) { return bars + 8u * (kStages + s); };
  auto empty_bar = [&](int s) { return bars + 8u * (2 * kStages + s); };
  auto accf_bar = [&](uint32_t b) { return bars + 8u * (3 * kStages + b); };
  auto acce_bar = [&](uint32_t b) { return bars + 8u * (3 * kStages + 2 + b); };
  const uint32_t done_bar = bars + 8u * (3 * kStages + 4);
  uint8_t* const tail = base_ptr + kStages * kStageBytes + 8 * kBars;
  uint32_t* const misc = reinterpret_cast<uint32_t*>(tail);            // TMEM address, present
  volatile float* const s_down = reinterpret_cast<float*>(misc + 2);   // [kScales], by block
  // [range][adapter] bytes: the 64-row blocks with the adapter; then, per 32 of
  // them, how many nonzero ones come before
  const int nmask = p.ranges * p.adapters;
  const int words = (nmask + kGroupMasks - 1) / kGroupMasks * (kGroupMasks / 4);
  uint32_t* const s_mask =
      reinterpret_cast<uint32_t*>(base_ptr + (kSmem - 1024 + 15) / 16 * 16);
  int* const s_prefix = reinterpret_cast<int*>(s_mask + words);
  const int warp = warp_id_uniform(), lane = static_cast<int>(lane_id());

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full_bar(s), 1u);
      mbar_init(tok_bar(s), 1u);
      mbar_init(empty_bar(s), 1u);
    }
    for (uint32_t b = 0; b < 2; ++b) {
      mbar_init(accf_bar(b), 2u);   // the products, and the MMA thread for the scale
      mbar_init(acce_bar(b), static_cast<uint32_t>(kEpi));
    }
    mbar_init(done_bar, 1u);
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(misc), kTmemCols);
    tmem_relinquish();
    griddep_launch_dependents();
  }
  for (int i = threadIdx.x; i < words; i += kThreads) s_mask[i] = 0u;
  __syncthreads();
  // ids is the caller's: nothing to wait for
  const int rows = min(p.M - p.row0, p.ranges * kRange);
  for (int i = threadIdx.x; i < rows; i += kThreads) {
    const int a = __ldg(p.ids + p.row0 + i);
    if (a >= 0 && a < p.adapters) {
      const int m = i / kRange * p.adapters + a;
      const uint32_t bit = 1u << (8 * (m & 3) + (i % kRange) / 64);
      if (!(reinterpret_cast<volatile uint32_t*>(s_mask)[m >> 2] & bit)) atomicOr(s_mask + (m >> 2), bit);
    }
  }
  __syncthreads();
  if (warp == 0) {
    int before = 0;
    const int groups = words / (kGroupMasks / 4);
    for (int g0 = 0; g0 < groups; g0 += 32) {
      int n = 0;
      if (g0 + lane < groups)
        for (int w = 0; w < kGroupMasks / 4; ++w)
          n += __popc(__vcmpgtu4(s_mask[(g0 + lane) * (kGroupMasks / 4) + w], 0u)) / 8;
      int incl = n;
      for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += v;
      }
      if (g0 + lane < groups) s_prefix[g0 + lane] = before + incl - n;
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) misc[1] = static_cast<uint32_t>(before);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = reinterpret_cast<volatile uint32_t*>(misc)[0];
  const int present = static_cast<int>(misc[1]);
  const uint8_t* const mask_bytes = reinterpret_cast<const uint8_t*>(s_mask);
  // the places of all masks, for the sum kernel; or, with one range, the
  // gradients of adapters without rows
  if (p.direct) {
    for (int a = 0; a < p.adapters; ++a) {
      if (mask_bytes[a]) continue;
      for (int src = 0; src < 2; ++src) {
        float* const o = src ? p.dB : p.dA;
        if (!o) continue;
        const long long n = 1ll * (src ? p.cols_g : p.cols_x) * p.R;
        for (long long i = blockIdx.x * kThreads + threadIdx.x; i < n; i += gridDim.x * kThreads)
          o[a * n + i] = p.beta != 0.0f ? p.beta * o[a * n + i] : 0.0f;
      }
    }
  }
  for (int m = blockIdx.x * kThreads + threadIdx.x; m < nmask && !p.direct;
       m += gridDim.x * kThreads) {
    int place = -1;
    if (mask_bytes[m]) {
      const int g = m / kGroupMasks;
      place = s_prefix[g];
      for (int i = g * kGroupMasks; i < m; ++i) place += mask_bytes[i] != 0;
    }
    p.table[m] = place;
  }
  griddep_wait();   // U and V
  const int all_tiles = p.tiles_x + p.tiles_g;
  const int per = all_tiles * p.chunks;
  const long long items = 1ll * present * per;
  auto item_at = [&](long long it) {
    Item t;
    t.present = static_cast<int>(it / per);
    const int v = static_cast<int>(it - 1ll * t.present * per);
    t.chunk = v / all_tiles;
    const int tile = v - t.chunk * all_tiles;
    t.src = tile < p.tiles_x ? 0 : 1;
    t.tile = t.src ? tile - p.tiles_x : tile;
    // the last group whose prefix does not pass the place, then within it
    int lo = 0, hi = words / (kGroupMasks / 4) - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (s_prefix[mid] <= t.present)
        lo = mid;
      else
        hi = mid - 1;
    }
    int left = t.present - s_prefix[lo], m = lo * kGroupMasks;
    for (;; ++m)
      if (mask_bytes[m] != 0 && left-- == 0) break;
    t.range = m / p.adapters;
    t.a = m - t.range * p.adapters;
    t.mask = mask_bytes[m];
    return t;
  };
  const unsigned long long limit = p.wait_limit_ns;
  DeviceStatus* const st = p.status;

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, issued = 0;
      bool ok = true;
      for (long long it = blockIdx.x; it < items && ok; it += gridDim.x) {
        const Item t = item_at(it);
        const int left = (t.src ? p.cols_g : p.cols_x) - t.tile * 256;
        const int boxes = min(4, (left + 63) / 64);
        const CUtensorMap* const tm = t.src ? &tmG : &tmX;
        for (int m = t.mask; m && ok; m &= m - 1) {
          const int row = p.row0 + t.range * kRange + (__ffs(m) - 1) * 64;
          if (!wait_parity(empty_bar(stage), phase ^ 1u, limit, st, 80)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(full_bar(stage), static_cast<uint32_t>(boxes * 8192 + kVBytes));
          tma_load_2d(base + stage * kStageBytes + kXBytes, t.src ? &tmV : &tmU, full_bar(stage),
                      64 * t.chunk, row);
          for (int b = 0; b < boxes; ++b)
            tma_load_2d(base + stage * kStageBytes + b * 8192, tm, full_bar(stage),
                        t.tile * 256 + b * 64, row);
          ++issued;
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      const uint32_t n = min(issued, static_cast<uint32_t>(kStages));
      for (uint32_t i = issued - n; i < issued; ++i)
        settle_wait(full_bar(static_cast<int>(i % kStages)), (i / kStages) & 1u, st, 81);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = make_idesc(0u, 128u, 64u, 1u, 1u);
      int stage = 0;
      uint32_t phase = 0, local = 0;
      bool ok = true;
      for (long long it = blockIdx.x; it < items && ok; it += gridDim.x) {
        const Item t = item_at(it);
        for (int m = t.mask; m; m &= m - 1) {
          const uint32_t buf = local & 1u;
          if (!wait_parity(acce_bar(buf), ((local >> 1) & 1u) ^ 1u, limit, st, 82) ||
              !wait_parity(full_bar(stage), phase, limit, st, 83) ||
              !wait_parity(tok_bar(stage), phase, limit, st, 84)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d0 = tmem + buf * 128;
          const uint32_t x0 = base + stage * kStageBytes, v0 = x0 + kXBytes;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t bd = smem_desc_sw128(v0 + kk * 2048, 8192u, 1024u);
            mma_f16_ss(d0, smem_desc_sw128(x0 + kk * 2048, 8192u, 1024u), bd, idesc, kk > 0);
            mma_f16_ss(d0 + 64, smem_desc_sw128(x0 + 16384 + kk * 2048, 8192u, 1024u), bd, idesc,
                       kk > 0);
          }
          mma_commit(empty_bar(stage));
          mma_commit(accf_bar(buf));
          mbar_arrive(accf_bar(buf));
          ++local;
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      mma_commit(done_bar);
      settle_wait(done_bar, 0u, st, 85);
    }
    __syncwarp();
  } else if (warp < 2 + kLoaders) {
    // Warp l of these takes the blocks l, l + 4, ... of the CTA's sequence, clears
    // the rows of other adapters (a lane has two rows) and hands on the scale of
    // the adapter's rows, which is that of the first of them.
    const int l = warp - 2;
    int stage = 0;
    uint32_t phase = 0, seq = 0;
    bool ok = true;
    for (long long it = blockIdx.x; it < items && ok; it += gridDim.x) {
      const Item t = item_at(it);
      for (int m = t.mask; m; m &= m - 1, ++seq) {
        if (static_cast<int>(seq & (kLoaders - 1)) == l) {
          const int row = p.row0 + t.range * kRange + (__ffs(m) - 1) * 64 + lane;
          const bool f0 = row < p.M && __ldg(p.ids + row) != t.a;
          const bool f1 = row + 32 < p.M && __ldg(p.ids + row + 32) != t.a;
          const bool mixed = __any_sync(0xffffffffu, f0 || f1);
          const unsigned int own0 = __ballot_sync(0xffffffffu, row < p.M && !f0);
          const unsigned int own1 = __ballot_sync(0xffffffffu, row + 32 < p.M && !f1);
          if (lane == 0)
            s_down[seq % kScales] =
                __ldg((t.src ? p.unscale_v : p.unscale_u) + row +
                      (own0 ? __ffs(own0) - 1 : 31 + __ffs(own1)));
          // a block of one adapter only passes through, but not before its stage
          // is free: two arrivals in one phase would hide one from the MMA warp
          if (lane == 0)
            ok = wait_parity(empty_bar(stage), phase ^ 1u, limit, st, 86) &&
                 (!mixed || wait_parity(full_bar(stage), phase, limit, st, 87));
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
          __syncwarp();
          if (!ok) break;
          if (mixed) {
            uint8_t* const sx = base_ptr + stage * kStageBytes;
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (i ? f1 : f0)
                for (int b = 0; b < 5; ++b)   // four boxes of X or dC, then U or V
#pragma unroll
                  for (int c = 0; c < 8; ++c)
                    *reinterpret_cast<uint4*>(sx + b * 8192 + (32 * i + lane) * 128 +
                                              (((c + lane) & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (lane == 0) mbar_arrive(tok_bar(stage));
        }
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else {
    const int quad = warp & 3, half = (warp - 2 - kLoaders) / 4;
    const bool vec_a = !p.direct || (reinterpret_cast<uintptr_t>(p.dA) & 15u) == 0;
    uint32_t local = 0;
    bool ok = true;
    for (long long it = blockIdx.x; it < items && ok; it += gridDim.x) {
      const Item t = item_at(it);
      float acc[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) acc[i] = 0.0f;
      for (int m = t.mask; m; m &= m - 1, ++local) {
        const uint32_t buf = local & 1u;
        if (!wait_parity(accf_bar(buf), (local >> 1) & 1u, limit, st, 88)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const float down = s_down[local % kScales];
        const uint32_t d0 =
            tmem + (static_cast<uint32_t>(32 * quad) << 16) + buf * 128 + half * 64;
        uint32_t hi[32], lo[32];
        tmem_ld_32x32b_x32(d0, hi);
        tmem_ld_32x32b_x32(d0 + 32, lo);
        tmem_wait_ld32(hi, lo);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acce_bar(buf));
#pragma unroll
        for (int i = 0; i < 32; ++i)
          acc[i] = fmaf(lora_join(__uint_as_float(hi[i]), __uint_as_float(lo[i])), down, acc[i]);
      }
      if (!ok) break;
      const int C = t.src ? p.cols_g : p.cols_x, r0 = 32 * t.chunk, nr = min(32, p.R - r0);
      const int c = t.tile * 256 + half * 128 + 32 * quad + lane;
      float* const out =
          p.direct ? (t.src ? p.dB : p.dA) + static_cast<long long>(t.a) * C * p.R
                   : p.part + t.present * p.part_stride + (t.src ? p.part_b : 0);
      if (c < C) {
        auto value = [&](float x, const float* old) {
          if (!p.direct) return x;
          return p.beta != 0.0f ? fmaf(p.alpha, x, p.beta * *old) : p.alpha * x;
        };
        if (t.src == 0 && p.R % 4 == 0 && vec_a) {
          // nr is a multiple of four: 16-byte stores along the ranks
          float* const o = out + static_cast<long long>(c) * p.R + r0;
#pragma unroll
          for (int r = 0; r < 32; r += 4)
            if (r < nr)
              __stcg(reinterpret_cast<float4*>(o + r),
                     make_float4(value(acc[r], o + r), value(acc[r + 1], o + r + 1),
                                 value(acc[r + 2], o + r + 2), value(acc[r + 3], o + r + 3)));
        } else {
#pragma unroll
          for (int r = 0; r < 32; ++r)
            if (r < nr) {
              float* const o = out + (t.src ? static_cast<long long>(r0 + r) * C + c
                                            : static_cast<long long>(c) * p.R + r0 + r);
              __stcg(o, value(acc[r], o));
            }
        }
      }
    }
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

// dA and dB := alpha * (the present ranges' partial sums in row order) + beta *
// themselves.
struct SumArgs {
  const float* part;
  long long part_stride, part_b, elems_a, elems_b;   // elements per adapter of dA, dB
  const int* table;
  float *dA, *dB;
  int adapters, ranges;
  float alpha, beta;
};

constexpr int kSumThreads = 256;

// One block per (1024 elements of a slice of dA or dB, adapter); four elements
// a thread, 256 apart.
__global__ void __launch_bounds__(kSumThreads) lora_outer_sum_kernel(const SumArgs p) {
  __shared__ int place[kSumThreads];   // present ranges, in order
  __shared__ int count;
  griddep_wait();
  const int a = blockIdx.y;
  const long long blocks_a = p.dA ? (p.elems_a + 4 * kSumThreads - 1) / (4 * kSumThreads) : 0;
  const int src = blockIdx.x < blocks_a ? 0 : 1;
  const long long e0 = (src ? blockIdx.x - blocks_a : blockIdx.x) * (4ll * kSumThreads) + threadIdx.x;
  const long long n = src ? p.elems_b : p.elems_a;
  const float* const part = p.part + (src ? p.part_b : 0);
  float s[4] = {};
  for (int r0 = 0; r0 < p.ranges; r0 += kSumThreads) {
    // a warp at a time keeps the places in row order
    if (threadIdx.x < 32) {
      int k = 0;
      for (int r = r0; r < min(p.ranges, r0 + kSumThreads); r += 32) {
        const int i = r + static_cast<int>(threadIdx.x);
        const int v = i < p.ranges ? p.table[i * p.adapters + a] : -1;
        const unsigned int m = __ballot_sync(0xffffffffu, v >= 0);
        if (v >= 0) place[k + __popc(m & ((1u << threadIdx.x) - 1u))] = v;
        k += __popc(m);
      }
      if (threadIdx.x == 0) count = k;
    }
    __syncthreads();
#pragma unroll 2
    for (int k = 0; k < count; ++k) {
      const float* q = part + place[k] * p.part_stride;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (e0 + j * kSumThreads < n) s[j] += __ldcg(q + e0 + j * kSumThreads);
    }
    __syncthreads();
  }
  float* const o = (src ? p.dB : p.dA) + a * n;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const long long e = e0 + j * kSumThreads;
    if (e < n) o[e] = p.beta != 0.0f ? fmaf(p.alpha, s[j], p.beta * o[e]) : p.alpha * s[j];
  }
}

// Ranges of one launch: the masks fit shared memory, the partial sums 2 GB.
int ranges_of(const LoraOuter& o) {
  const long long per = 4ll * std::min(o.adapters, kRange) * o.R * (o.K + o.N);
  const long long fit = std::min<long long>(kMaxMasks / std::max(1, o.adapters),
                                            (2ll << 30) / std::max(1ll, per));
  return static_cast<int>(
      std::max(1ll, std::min<long long>((o.M + kRange - 1) / kRange, fit)));
}

}  // namespace

size_t lora_outer_bytes(const LoraOuter& o) {
  if (o.M <= kRange) return 0;
  const long long ranges = ranges_of(o);
  return lora_round256(4 * static_cast<size_t>(ranges) * o.adapters) +
         4 * static_cast<size_t>(ranges) * std::min(o.adapters, kRange) * o.R *
             (static_cast<size_t>(o.K) + o.N);
}

int lora_outer(const LoraOuter& o, void* scratch, const LoraDevice& d, cudaStream_t stream) {
  if (o.adapters > kMaxMasks) return GEMM_ERR_ARG;
  CUtensorMap tmX{}, tmG{};
  if (o.dA)
    if (int rc = encode_map_f16(&tmX, o.X, o.M, o.K, o.ldx, 64, 64)) return rc;
  if (o.dB)
    if (int rc = encode_map_f16(&tmG, o.G, o.M, o.N, o.ldg, 64, 64)) return rc;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return GEMM_ERR_CUDA;
  static bool configured[64] = {};
  if (dev < 64 && !configured[dev]) {
    if (cudaFuncSetAttribute(lora_outer_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             232448) != cudaSuccess)
      return GEMM_ERR_CUDA;
    configured[dev] = true;
  }
  const int ranges = ranges_of(o);
  Args a{};
  CUtensorMap tmU{}, tmV{};
  const int chunks = (o.R + 31) / 32;
  if (o.dA) {
    if (int rc = encode_map_f16(&tmU, o.U->scaled, o.M, 64 * chunks, 64ll * chunks, 64, 64)) return rc;
    a.unscale_u = o.U->unscale;
  }
  if (o.dB) {
    if (int rc = encode_map_f16(&tmV, o.V->scaled, o.M, 64 * chunks, 64ll * chunks, 64, 64)) return rc;
    a.unscale_v = o.V->unscale;
  }
  a.cols_x = o.K;
  a.cols_g = o.N;
  a.tiles_x = o.dA ? (o.K + 255) / 256 : 0;
  a.tiles_g = o.dB ? (o.N + 255) / 256 : 0;
  a.ids = o.ids;
  a.M = o.M;
  a.R = o.R;
  a.adapters = o.adapters;
  a.chunks = chunks;
  a.table = static_cast<int*>(scratch);   // unused, like part, when direct
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(scratch) +
                                    lora_round256(4 * static_cast<size_t>(ranges) * o.adapters));
  a.part_b = 1ll * o.K * o.R;
  a.part_stride = a.part_b + 1ll * o.R * o.N;
  a.wait_limit_ns = d.wait_limit_ns;
  a.status = d.status;
  a.dA = o.dA;
  a.dB = o.dB;
  a.alpha = o.alpha;
  a.beta = o.beta;
  a.direct = o.M <= kRange;
  SumArgs s{};
  s.part = a.part;
  s.part_stride = a.part_stride;
  s.part_b = a.part_b;
  s.elems_a = 1ll * o.K * o.R;
  s.elems_b = 1ll * o.R * o.N;
  s.table = a.table;
  s.dA = o.dA;
  s.dB = o.dB;
  s.adapters = o.adapters;
  s.alpha = o.alpha;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  for (int r0 = 0; r0 * kRange < o.M; r0 += ranges) {
    a.row0 = r0 * kRange;
    a.ranges = std::min(ranges, (o.M + kRange - 1) / kRange - r0);
    const int nmask = a.ranges * o.adapters;
    const int words = (nmask + kGroupMasks - 1) / kGroupMasks * (kGroupMasks / 4);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(d.sms), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmem + 16 + 4 * static_cast<size_t>(words + words / (kGroupMasks / 4));
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = r0 == 0 ? 1 : 0;   // a later slab waits for the sums of the one before
    if (counted_launch(cudaLaunchKernelEx(&cfg, lora_outer_kernel, tmX, tmG, tmU, tmV, a)) != cudaSuccess)
      return GEMM_ERR_CUDA;
    if (a.direct) return GEMM_OK;
    s.ranges = a.ranges;
    s.beta = r0 == 0 ? o.beta : 1.0f;
    const long long blocks =
        (s.dA ? (s.elems_a + 4 * kSumThreads - 1) / (4 * kSumThreads) : 0) +
        (s.dB ? (s.elems_b + 4 * kSumThreads - 1) / (4 * kSumThreads) : 0);
    if (blocks > 0x7fffffff) return GEMM_ERR_ARG;
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(o.adapters), 1);
    cfg.blockDim = dim3(kSumThreads, 1, 1);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    if (counted_launch(cudaLaunchKernelEx(&cfg, lora_outer_sum_kernel, s)) != cudaSuccess)
      return GEMM_ERR_CUDA;
  }
  return GEMM_OK;
}

}  // namespace gb300
