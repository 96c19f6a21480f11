// lora_shrink.cu -- the low-rank products V = s X A[a] (and, for gradients,
// U = s dC B[a]^T) of many rows on the tensor cores, with what the kernels
// after it need: each 256-row block's distinct adapters, and which adapters
// hold weights that are not finite.
//
// One CTA per (128 rows, K slice): the rows of x are the M operand, the
// adapters that occur among them the N operand, RP columns each (the rank
// rounded up to 16, 32, 64 or 128), a few of them at a time; a row keeps the
// columns of its own adapter.  What binds is reading x once: 2 R
// multiply-adds per half, where the tensor cores take ~280.  The K slices of a
// tile are a cluster: each leaves its partial sums in its own shared memory and
// adds up its share of the rows from all of them, in slice order (through global
// memory and a counter, the last slice alone took 8 us to add up eight).  The
// same step writes V as the tensor cores take it: two halves per entry, hi + lo
// (22 significant bits or 2^-25), 32 ranks' hi and then their lo as 64 columns, so that
// the kernels after this one load it by TMA.  For C and dX these share an
// accumulator with the rest of the product and so have no scale: a row with an
// entry past the half range has zeros instead, a mark, and is added in fp32 from V.
// One whose largest entry is below 2^-11 (2^-25 is more than 2^-14 of it) is marked
// as well: what its halves leave out matters, and is added, only where weights are
// large.  alpha times the sum over R ranks is then off by about alpha sqrt(R) max|F|
// 2^-25, which is below the result's own rounding while alpha sqrt(R) max|F| <= 1.
// For the adapters' gradients it is
// first scaled, each adapter of the 128 rows by itself, by the power of two that
// brings its largest finite magnitude into [2^13, 2^14): gradients of any size
// keep their bits, whatever the rows of other adapters hold.
//
// The tensor cores truncate when they add to an fp32 accumulator, by up to
// 2^-23 of it per 16 products of K, always toward zero.  The gradients of the
// adapters are fp32, so a run of 128 products of K is the longest that stays in
// TMEM; the runs are added up in registers, rounded to nearest.
//
// F[a] is stored along K (C x R: MN-major N operand) for V, or along the ranks
// (R x C: K-major) for U.  Along K a rank of 16 or 32 is staged as rows of 32 or
// 64 bytes: in 128-byte rows, mostly padding, only two stages fitted beside four
// adapters.
#include "lora.h"

namespace gb300 {
namespace {

constexpr int kThreads = 192;                // TMA, MMA, 4 epilogue warps
constexpr int kMaxStages = 6;
constexpr int kMaxSlices = 8;                // a portable cluster
constexpr int kXBytes = 128 * 128;           // 128 rows of a k-block
constexpr int kFoldKb = 2;                   // k-blocks accumulated in TMEM

struct Args {
  LoraShrinkJob job[2];
  int njobs;
  const int* ids;
  const float* scales;
  int M, R, adapters, ldv;
  int* lists;             // [256-row block][kLoraListStride]
  int* bad;               // [adapters][kLoraBadParts]
  const uint16_t* check;  // weights to look for non-finite ones in, rows x cols each
  long long ld_check, check_stride;
  int check_rows, check_cols;
  uint32_t large;         // twice: bits of the largest half that is not large
  // blocks: items of the first job, of the second, lists, checks (the short ones
  // last: items start one to an SM)
  int first_item, first_list, first_check;
  int slices, kb[2];
  int ring;               // bytes of the operand ring: twice as many when every
                          // CTA can have an SM for itself
  int chunks;             // of 32 ranks
  unsigned long long wait_limit_ns;
  DeviceStatus* status;
};

// The distinct adapters of ids[0, n), n <= 256, in order of first occurrence
// within and among runs of 32 rows into `list`; returns their number.  slot[i]:
// place of row i's adapter, -1 for none.  All kThreads threads; `first` has
// room for 256 words, `cnt` for 10.
__device__ int distinct(const int* ids, int n, int adapters, int* list, int* slot, int* first,
                        int* cnt) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int runs = (n + 31) / 32;
  // every run by itself: its adapters and how many, each row's place among them
  for (int g = warp; g < runs; g += kThreads / 32) {
    const int i = 32 * g + lane;
    int a = i < n ? __ldg(ids + i) : -1;
    if (a >= adapters) a = -1;
    const unsigned int same = __match_any_sync(0xffffffffu, a);
    const unsigned int heads =
        __ballot_sync(0xffffffffu, a >= 0 && (same & ((1u << lane) - 1u)) == 0u);
    const int head = __ffs(same) - 1;
    if (i < n) slot[i] = a < 0 ? -1 : __popc(heads & ((1u << head) - 1u));
    if (heads >> lane & 1u) first[32 * g + __popc(heads & ((1u << lane) - 1u))] = a;
    if (lane == 0) cnt[1 + g] = __popc(heads);
  }
  __syncthreads();
  // one warp joins the runs: run g's adapters (a lane each) against the list so far
  if (warp == 0) {
    int total = 0;
    for (int g = 0; g < runs; ++g) {
      const int a = lane < cnt[1 + g] ? first[32 * g + lane] : -1;
      int at = -1;
      for (int k = 0; k < total; ++k)
        if (list[k] == a) at = k;
      const unsigned int fresh = __ballot_sync(0xffffffffu, a >= 0 && at < 0);
      if (a >= 0) {
        if (at < 0) {
          at = total + __popc(fresh & ((1u << lane) - 1u));
          list[at] = a;
        }
        first[32 * g + lane] = at;
      }
      total += __popc(fresh);
      __syncwarp();
    }
    if (lane == 0) cnt[0] = total;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads)
    if (slot[i] >= 0) slot[i] = first[(i & ~31) + slot[i]];
  __syncthreads();
  return cnt[0];
}

// RP: columns of an adapter.
template <int RP>
struct Cfg {
  static constexpr int kCols = RP > 64 ? RP : 64;      // columns of a pass: whole adapters
  static constexpr int kGroup = kCols / RP;            // most adapters per pass
  static constexpr int kNBytes = 128 * RP;             // an adapter's k-block
  static constexpr int kTmemCols = 2 * kCols;
  // operand ring and the tile's partial sums: two CTAs fit on an SM up to rank 64
  static constexpr int kRing = RP > 32 ? 65536 : 81920;
  static constexpr int kSums = 128 * RP * 4;
  static constexpr int kSmem = kSums + 1024 + 8 * (2 * kMaxStages + 5) + 16;   // beside it
  static_assert(kRing / (kXBytes + kNBytes) >= 2, "two stages");
  static_assert(kRing >= kSums, "the ring holds the tile's sums");
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ float ld_cluster_f(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

template <int RP>
__global__ void __launch_bounds__(kThreads, 2)
    lora_shrink_tc_kernel(const __grid_constant__ CUtensorMap tmX0,
                          const __grid_constant__ CUtensorMap tmF0,
                          const __grid_constant__ CUtensorMap tmX1,
                          const __grid_constant__ CUtensorMap tmF1, const Args p) {
  using G = Cfg<RP>;
  __shared__ int s_first[256], s_list[256], s_slot[256], s_cnt[10];
  __shared__ unsigned int s_top[128];   // by slot: largest finite magnitude
  if (threadIdx.x == 0) {
    prefetch_tensormap(&tmX0);
    prefetch_tensormap(&tmF0);
    if (p.njobs > 1) {
      prefetch_tensormap(&tmX1);
      prefetch_tensormap(&tmF1);
    }
  }
  const int b = blockIdx.x;
  if (b >= p.first_list) griddep_launch_dependents();
  if (b >= p.first_check) {
    // ---- a quarter of an adapter (if a row uses it): are its weights finite, are
    // some large
    const int check = b - p.first_check, adapter = check / kLoraBadParts;
    if (adapter >= p.adapters) return;   // fills up the last cluster
    bool used = false;
#pragma unroll 16
    for (int i = threadIdx.x; i < p.M; i += kThreads) used |= __ldg(p.ids + i) == adapter;
    int bad = 0;
    unsigned int big = 0u;
    if (__syncthreads_or(used)) {
      const uint16_t* f = p.check + static_cast<long long>(adapter) * p.check_stride;
      const int groups = (p.check_cols + 7) / 8, part = check - adapter * kLoraBadParts;
      const int end = static_cast<int>((part + 1ll) * p.check_rows / kLoraBadParts);
      // thread t takes 16-byte pieces t, t + kThreads, ... of the rows' pieces
      int r = static_cast<int>(1ll * part * p.check_rows / kLoraBadParts) + threadIdx.x / groups;
      int g = threadIdx.x % groups;
      const int dr = kThreads / groups, dg = kThreads % groups;
#pragma unroll 16
      for (; r < end; r += dr + (g + dg >= groups), g += g + dg >= groups ? dg - groups : dg) {
        const int c = 8 * g;
        const uint16_t* q = f + static_cast<long long>(r) * p.ld_check + c;
        if (c + 8 <= p.check_cols) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(q));
          // an exponent of all ones in either half
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            bad |= __vcmpgeu2(w[j] & 0x7FFF7FFFu, 0x7C007C00u) != 0u;
            big |= __vcmpgtu2(w[j] & 0x7FFF7FFFu, p.large);
          }
        } else {
          for (int j = 0; c + j < p.check_cols; ++j) {
            bad |= (q[j] & 0x7FFFu) >= 0x7C00u;
            big |= (q[j] & 0x7FFFu) > (p.large & 0xFFFFu);
          }
        }
      }
    }
    bad = __syncthreads_or(bad);
    big = __syncthreads_or(big != 0u);
    if (threadIdx.x == 0) p.bad[check] = (bad ? 1 : 0) | (big ? 2 : 0);
    return;
  }
  if (b >= p.first_list) {
    // ---- the distinct adapters of a 256-row block
    const int blk = b - p.first_list, row0 = blk * 256;
    const int n = distinct(p.ids + row0, min(256, p.M - row0), p.adapters, s_list, s_slot, s_first,
                           s_cnt);
    int* const out = p.lists + static_cast<long long>(blk) * kLoraListStride;
    for (int i = threadIdx.x; i < n; i += kThreads) out[1 + i] = s_list[i];
    if (threadIdx.x == 0) out[0] = n;
    return;
  }
  // ---- a product: rows [row0, row0 + 128), one K slice
  const int which = b >= p.first_item ? 1 : 0;
  const LoraShrinkJob& job = p.job[which];
  const CUtensorMap* const tmX = which ? &tmX1 : &tmX0;
  const CUtensorMap* const tmF = which ? &tmF1 : &tmF0;
  const int item = b - which * p.first_item, slices = p.slices;
  const int tile = item / slices, slice = item - tile * slices;
  const int row0 = tile * 128, rows = min(128, p.M - row0);
  const int kb0 = slice * p.kb[which] / slices, kb1 = (slice + 1) * p.kb[which] / slices;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const base_ptr = smem_raw + (base - raw);
  const uint32_t bars = base + p.ring + G::kSums;
  auto full_bar = [&](int s) { return bars + 8u * s; };
  auto empty_bar = [&](int s) { return bars + 8u * (kMaxStages + s); };
  auto accf_bar = [&](uint32_t i) { return bars + 8u * (2 * kMaxStages + i); };
  auto acce_bar = [&](uint32_t i) { return bars + 8u * (2 * kMaxStages + 2 + i); };
  const uint32_t done_bar = bars + 8u * (2 * kMaxStages + 4);
  float* const sums = reinterpret_cast<float*>(base_ptr + p.ring);   // [128][ldv]
  uint8_t* const tmem_ptr = base_ptr + p.ring + G::kSums + 8 * (2 * kMaxStages + 5);
  const int warp = warp_id_uniform(), lane = static_cast<int>(lane_id());
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(full_bar(s), 1u);
      mbar_init(empty_bar(s), 1u);
    }
    for (uint32_t i = 0; i < 2; ++i) {
      mbar_init(accf_bar(i), 1u);
      mbar_init(acce_bar(i), 4u);
    }
    mbar_init(done_bar, 1u);
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(tmem_ptr), G::kTmemCols);
    tmem_relinquish();
    // only now: the next kernel holds its tensor memory until this one ends
    griddep_launch_dependents();
  }
  if (job.scaled && threadIdx.x < 128) s_top[threadIdx.x] = 0u;
  const int n = distinct(p.ids + row0, rows, p.adapters, s_list, s_slot, s_first, s_cnt);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_ptr);
  // adapters of a pass: as many as leave the ring two stages; a stage holds the
  // rows and as many adapters as a pass can have here
  const int group = min(min(max(n, 1), G::kGroup), (p.ring / 2 - kXBytes) / G::kNBytes);
  const int passes = (n + group - 1) / group;
  const uint32_t stage_bytes = kXBytes + group * G::kNBytes;
  const int S = min(kMaxStages, static_cast<int>(p.ring / stage_bytes));
  const unsigned long long limit = p.wait_limit_ns;
  DeviceStatus* const st = p.status;
  const int fboxes = job.k_major ? 1 : (p.R + 63) / 64;
  const uint32_t fbytes = job.k_major || RP <= 64 ? RP * 128u : fboxes * 8192u;

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, issued = 0;
      bool ok = true;
      for (int ps = 0; ps < passes && ok; ++ps) {
        const int g0 = ps * group, gn = min(group, n - g0);
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!wait_parity(empty_bar(stage), phase ^ 1u, limit, st, 70)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(full_bar(stage), kXBytes + gn * fbytes);
          const uint32_t dst = base + stage * stage_bytes;
          tma_load_2d(dst, tmX, full_bar(stage), kb * 64, row0);
          for (int j = 0; j < gn; ++j) {
            const uint32_t f = dst + kXBytes + j * G::kNBytes;
            if (job.k_major) {
              tma_load_3d(f, tmF, full_bar(stage), kb * 64, 0, s_list[g0 + j]);
            } else {
              for (int c = 0; c < fboxes; ++c)
                tma_load_3d(f + c * 8192, tmF, full_bar(stage), 64 * c, kb * 64, s_list[g0 + j]);
            }
          }
          ++issued;
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      const uint32_t left = min(issued, static_cast<uint32_t>(S));
      for (uint32_t i = issued - left; i < issued; ++i)
        settle_wait(full_bar(static_cast<int>(i % S)), (i / S) & 1u, st, 71);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = make_idesc(0u, 128u, RP, 0u, job.k_major ? 0u : 1u);
      int stage = 0;
      uint32_t phase = 0, local = 0;
      bool ok = true;
      for (int ps = 0; ps < passes && ok; ++ps) {
        const int gn = min(group, n - ps * group);
        for (int k0 = kb0; k0 < kb1 && ok; k0 += kFoldKb) {
          const uint32_t buf = local & 1u;
          if (!wait_parity(acce_bar(buf), ((local >> 1) & 1u) ^ 1u, limit, st, 72)) {
            ok = false;
            break;
          }
          tc_fence_after();
          for (int kb = k0; kb < min(kb1, k0 + kFoldKb); ++kb) {
            if (!wait_parity(full_bar(stage), phase, limit, st, 73)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t x0 = base + stage * stage_bytes, f0 = x0 + kXBytes;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const uint64_t ad = smem_desc_sw128(x0 + kk * 32, 16u, 1024u);
              for (int j = 0; j < gn; ++j) {
                const uint32_t f = f0 + j * G::kNBytes;
                mma_f16_ss(tmem + buf * G::kCols + j * RP, ad,
                           job.k_major ? smem_desc_sw128(f + kk * 32, 16u, 1024u)
                           : RP == 16  ? smem_desc_sw32(f + kk * 512, 2048u, 256u)
                           : RP == 32  ? smem_desc_sw64(f + kk * 1024, 4096u, 512u)
                                       : smem_desc_sw128(f + kk * 2048, 8192u, 1024u),
                           idesc, (kb > k0 || kk > 0) ? 1u : 0u);
              }
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
        }
      }
      mma_commit(done_bar);
      settle_wait(done_bar, 0u, st, 74);
    }
    __syncwarp();
  } else {
    const int quad = warp & 3, lr = 32 * quad + lane;   // this thread's row of the tile
    const bool in = lr < rows;
    const int slot = in ? s_slot[lr] : -1;
    float* const out = sums + lr * p.ldv;
    if (slot < 0)
      for (int r = 0; r < p.ldv; r += 4)
        *reinterpret_cast<float4*>(out + r) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    uint32_t local = 0;
    bool ok = true;
    for (int ps = 0; ps < passes && ok; ++ps) {
      float acc[G::kCols];
#pragma unroll
      for (int i = 0; i < G::kCols; ++i) acc[i] = 0.0f;
      for (int k0 = kb0; k0 < kb1; k0 += kFoldKb, ++local) {
        const uint32_t buf = local & 1u;
        if (!wait_parity(accf_bar(buf), (local >> 1) & 1u, limit, st, 75)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d0 = tmem + (static_cast<uint32_t>(32 * quad) << 16) + buf * G::kCols;
#pragma unroll
        for (int c = 0; c < G::kCols; c += 16) {
          uint32_t g[8], h[8];
          tmem_ld_32x32b_x8(d0 + c, g);
          tmem_ld_32x32b_x8(d0 + c + 8, h);
          tmem_wait_ld2(g, h);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            acc[c + i] += __uint_as_float(g[i]);
            acc[c + 8 + i] += __uint_as_float(h[i]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acce_bar(buf));
      }
      if (!ok) break;
      const int mine = slot - ps * group;
      if (slot >= 0 && mine >= 0 && mine < group) {
        const float s = p.scales ? p.scales[s_list[slot]] : 1.0f;
#pragma unroll
        for (int j = 0; j < G::kGroup; ++j)
          if (mine == j)
#pragma unroll
            for (int r = 0; r < RP; r += 4)
              if (r < p.ldv) {
                // the ranks past R are products with zeros, which an Inf or NaN
                // of x makes NaN
                auto value = [&](int i) { return i < p.R ? s * acc[j * RP + i] : 0.0f; };
                *reinterpret_cast<float4*>(out + r) =
                    make_float4(value(r), value(r + 1), value(r + 2), value(r + 3));
              }
      }
    }
  }
  __syncwarp();
  cluster_sync();   // every slice's sums are in its shared memory; its ring is idle
  // this CTA's share of the tile's rows: the slices added up in order
  const int share = 128 / slices, r0 = slice * share;
  const int per = p.ldv / 4, total = max(0, min(share, rows - r0)) * per;
  float4* const mine = reinterpret_cast<float4*>(base_ptr);   // [share][ldv]
  float4* const vout =
      reinterpret_cast<float4*>(job.V + (static_cast<long long>(row0) + r0) * p.ldv);
  const uint32_t sums_addr = base + p.ring + r0 * p.ldv * 4;
  for (int i = threadIdx.x; i < total; i += kThreads) {
    float4 t[kMaxSlices];
#pragma unroll
    for (int k = 0; k < kMaxSlices; ++k)
      if (k < slices) t[k] = ld_cluster_f4(map_to_cta(sums_addr + 16 * i, k));
    float4 v = t[0];
#pragma unroll
    for (int k = 1; k < kMaxSlices; ++k)
      if (k < slices) {
        v.x += t[k].x;
        v.y += t[k].y;
        v.z += t[k].z;
        v.w += t[k].w;
      }
    mine[i] = v;
    vout[i] = v;
  }
  int* const s_exp = s_first;   // by slot: the exponent of its scale
  if (job.scaled) {
    for (int i = threadIdx.x; i < total; i += kThreads) {   // this thread's own
      const int slot = s_slot[r0 + i / per];
      if (slot >= 0) atomicMax(s_top + slot, lora_top_bits(mine[i]));
    }
    __syncwarp();
    cluster_sync();   // every slice's largest magnitudes are known
    for (int i = threadIdx.x; i < n; i += kThreads) {
      float t[kMaxSlices], top = 0.0f;
#pragma unroll
      for (int k = 0; k < kMaxSlices; ++k)
        t[k] = k < slices ? ld_cluster_f(map_to_cta(smem_addr(s_top + i), k)) : 0.0f;
#pragma unroll
      for (int k = 0; k < kMaxSlices; ++k) top = fmaxf(top, t[k]);
      s_exp[i] = lora_scale_exponent(top);
    }
  }
  __syncthreads();
  if (job.packed || job.scaled) {
    // eight threads a row and chunk, four ranks each
    const int q = threadIdx.x & 7, nrow = total / per;
    for (int i = threadIdx.x >> 3; i < nrow * p.chunks; i += kThreads / 8) {
      const int r = i / p.chunks, c = i - r * p.chunks, piece = 8 * c + q;
      const float4 v =
          piece < per ? mine[r * per + piece] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      const long long o =
          ((static_cast<long long>(row0) + r0 + r) * p.chunks + c) * 64 + 4 * q;
      if (job.packed) {
        // the row's largest finite magnitude, by the eight threads
        unsigned int top = 0u;
        for (int j = q; j < per; j += 8) top = max(top, lora_top_bits(mine[r * per + j]));
        for (int d = 4; d; d >>= 1)
          top = max(top, __shfl_xor_sync(0xFFu << (lane & 24), top, d));
        const float t = __uint_as_float(top);
        const bool past = t >= 65520.0f;   // rounds to infinity
        lora_store_split(job.packed + o, past ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : v);
        if (c == 0 && q == 0)
          job.apart[row0 + r0 + r] = past ? 1 : (t > 0.0f && t < 0x1p-11f ? 2 : 0);
      }
      if (job.scaled) {
        const int slot = s_slot[r0 + r], e = slot < 0 ? 0 : s_exp[slot];
        const float up = lora_power(e);
        lora_store_split(job.scaled + o, make_float4(up * v.x, up * v.y, up * v.z, up * v.w));
        if (c == 0 && q == 0) job.unscale[row0 + r0 + r] = lora_power(-e);
      }
    }
  }
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, G::kTmemCols);
  // no CTA leaves while another may still read its shared memory
  __syncwarp();
  cluster_sync();
}

template <int RP>
int launch(const CUtensorMap* maps, Args a, int grid, int sms, cudaStream_t stream) {
  a.ring = grid <= sms ? 2 * Cfg<RP>::kRing : Cfg<RP>::kRing;
  static_assert(2 * Cfg<RP>::kRing + Cfg<RP>::kSmem <= 232448, "shared memory budget");
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return GEMM_ERR_CUDA;
  static bool configured[64] = {};
  if (dev < 64 && !configured[dev]) {
    if (cudaFuncSetAttribute(lora_shrink_tc_kernel<RP>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             2 * Cfg<RP>::kRing + Cfg<RP>::kSmem) != cudaSuccess)
      return GEMM_ERR_CUDA;
    configured[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(a.ring) + Cfg<RP>::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(a.slices);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, lora_shrink_tc_kernel<RP>, maps[0], maps[1],
                                           maps[2], maps[3], a);
  return counted_launch(e) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

// K slices of a tile: with them the CTAs of all jobs, checks and lists about
// fill the two places an SM has, at least two k-blocks a slice for the longer
// job (slices of the other may be empty, and its CTAs count by their length: 1949
// x 384 x 5568 of rank 24, 24 adapters, 96 -> 92 us).  Counted for all the jobs that
// the operator can have, so that a gradient asked for alone has the bits it has
// beside the others.
int slices_of(const LoraShrinkPlan& p, int sms) {
  const int tiles = (p.M + 127) / 128;
  const long long extra = 1ll * kLoraBadParts * p.adapters + (p.M + 255) / 256;
  const long long room = std::max<long long>((p.R > 64 ? 1 : 2) * sms - extra, sms);
  int s = 1;
  while (2 * s <= kMaxSlices && 2 * s * tiles * p.sum_c <= room * p.max_c &&
         4 * s <= (p.max_c + 63) / 64)
    s *= 2;
  return s;
}

}  // namespace

size_t lora_shrink_bytes(const LoraShrinkPlan& p) {
  size_t n = lora_round256(4 * static_cast<size_t>((p.M + 255) / 256) * kLoraListStride) +
             lora_round256(4 * kLoraBadParts * static_cast<size_t>(p.adapters));
  for (int j = 0; j < p.njobs; ++j) {
    n += lora_round256(4 * static_cast<size_t>(p.M) * p.ldv);
    const size_t packed = lora_round256(2 * 64 * static_cast<size_t>((p.R + 31) / 32) * p.M);
    if (p.job[j].want & kLoraPacked) n += packed + lora_round256(p.M);
    if (p.job[j].want & kLoraScaled)
      n += packed + lora_round256(4 * static_cast<size_t>(p.M));
  }
  return n;
}

int lora_shrink(LoraShrinkPlan& p, void* scratch, const LoraDevice& d, cudaStream_t stream) {
  uint8_t* buf = static_cast<uint8_t*>(scratch);
  auto take = [&](size_t bytes) {
    uint8_t* const q = buf;
    buf += lora_round256(bytes);
    return q;
  };
  const int tiles = (p.M + 127) / 128, blocks = (p.M + 255) / 256;
  const int rp = p.R <= 16 ? 16 : (p.R <= 32 ? 32 : (p.R <= 64 ? 64 : 128));
  Args a{};
  a.njobs = p.njobs;
  a.ids = p.ids;
  a.scales = p.scales;
  a.M = p.M;
  a.R = p.R;
  a.adapters = p.adapters;
  a.ldv = p.ldv;
  a.chunks = (p.R + 31) / 32;
  p.lists = reinterpret_cast<int*>(take(4 * static_cast<size_t>(blocks) * kLoraListStride));
  p.bad = reinterpret_cast<int*>(take(4 * kLoraBadParts * static_cast<size_t>(p.adapters)));
  a.lists = p.lists;
  a.bad = p.bad;
  a.check = p.check;
  a.ld_check = p.ld_check;
  a.check_stride = p.check_stride;
  a.check_rows = p.check_rows;
  a.check_cols = p.check_cols;
  const uint32_t large = __half_as_ushort(__float2half_rz(std::min(p.large, 65504.0f)));
  a.large = large * 0x10001u;
  a.wait_limit_ns = d.wait_limit_ns;
  a.status = d.status;
  a.slices = slices_of(p, d.sms);
  a.first_item = tiles * a.slices;
  a.first_list = p.njobs * a.first_item;
  a.first_check = a.first_list + (p.check ? blocks : 0);
  int grid = a.first_check + (p.check ? kLoraBadParts * p.adapters : 0);
  grid = (grid + a.slices - 1) / a.slices * a.slices;   // whole clusters
  CUtensorMap maps[4] = {};
  for (int j = 0; j < p.njobs; ++j) {
    LoraShrinkJob& job = p.job[j];
    job.tiles = tiles;
    a.kb[j] = (job.C + 63) / 64;
    job.V = reinterpret_cast<float*>(take(4 * static_cast<size_t>(p.M) * p.ldv));
    const size_t packed = 2 * 64 * static_cast<size_t>((p.R + 31) / 32) * p.M;
    if (job.want & kLoraPacked) {
      job.packed = reinterpret_cast<uint16_t*>(take(packed));
      job.apart = take(static_cast<size_t>(p.M));
    }
    if (job.want & kLoraScaled) {
      job.scaled = reinterpret_cast<uint16_t*>(take(packed));
      job.unscale = reinterpret_cast<float*>(take(4 * static_cast<size_t>(p.M)));
    }
    if (int rc = encode_map_f16(&maps[2 * j], job.x, p.M, job.C, job.ldx, 64, 128)) return rc;
    if (int rc = job.k_major ? encode_map_f16_stack(&maps[2 * j + 1], job.F, p.R, job.C, job.ldf,
                                                    p.adapters, job.f_stride, 64, rp)
                             : encode_map_f16_stack(&maps[2 * j + 1], job.F, job.C, p.R, job.ldf,
                                                    p.adapters, job.f_stride, std::min(rp, 64), 64,
                                                    2 * std::min(rp, 64)))
      return rc;
    a.job[j] = job;
  }
  switch (rp) {
    case 16: return launch<16>(maps, a, grid, d.sms, stream);
    case 32: return launch<32>(maps, a, grid, d.sms, stream);
    case 64: return launch<64>(maps, a, grid, d.sms, stream);
    default: return launch<128>(maps, a, grid, d.sms, stream);
  }
}

}  // namespace gb300
