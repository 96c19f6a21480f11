// lora_rows.cu -- the low-rank products V = s x F[a] row by row on CUDA cores:
// each row reads its own adapter, 2 C R bytes from L2, whatever the other rows
// have.  For decoding batches this hides behind the stream of W; for the
// gradients of a few rows over many adapters it replaces the tensor-core shrink
// (lora_shrink.cu), which passes once over its rows for every few adapters among
// them (dA, dB and dX of 49 rows over 29 adapters of rank 32, 4096 x 4096: 105 us that
// way, 41 this way).
//
//   lora_rows_kernel  (row, K slice, job): F[a] stored along K (thread (k, v):
//                     ranks 8v .. 8v + 7 of row k) or along the ranks (a warp
//                     per rank, 16-byte pieces of its row)
//   lora_pack_kernel  (128 rows, job): the slices added up in order, and V as
//                     lora_shrink.cu writes it for the gradient kernel
#include "lora.h"

namespace gb300 {
namespace {

constexpr int kThreads = 256;

// FORWARD: one job, stored along the ranks (0.3 us less than found at run time).
template <bool FORWARD>
__global__ void __launch_bounds__(kThreads) lora_rows_kernel(const LoraRows p) {
  __shared__ float red[kThreads * 9];
  __shared__ float red2[kThreads];
  griddep_launch_dependents();
  const int per_job = p.M * p.slices;
  const int which = !FORWARD && static_cast<int>(blockIdx.x) >= per_job ? 1 : 0;
  const int item = blockIdx.x - which * per_job;
  const LoraRowsJob job = which ? p.job[1] : p.job[0];
  const int i = item / p.slices, slice = item - i * p.slices;
  const int a = __ldg(p.ids + i);
  float* const out = job.V + (static_cast<long long>(i) * p.slices + slice) * p.R;
  if (a < 0 || a >= p.adapters) {
    for (int r = threadIdx.x; r < p.R; r += kThreads) out[r] = 0.0f;
    return;
  }
  const float scale = p.scales ? p.scales[a] : 1.0f;
  const uint16_t* const x = job.x + static_cast<long long>(i) * job.ldx;
  const uint16_t* const f = job.F + static_cast<long long>(a) * job.f_stride;
  // slices of multiples of eight columns, so that 16-byte pieces stay whole
  const int len = ((job.C + p.slices - 1) / p.slices + 7) / 8 * 8;
  const int k0 = min(job.C, slice * len), k1 = min(job.C, k0 + len);
  if (!FORWARD && job.k_major) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int r = warp; r < p.R; r += kThreads / 32) {
      const uint16_t* const fr = f + static_cast<long long>(min(r, job.ranks - 1)) * job.ldf;
      float s = 0.0f;
#pragma unroll 2
      for (int k = k0 + 8 * lane; k < k1; k += 256) {
        if (k + 8 <= k1) {
          const uint4 u = __ldg(reinterpret_cast<const uint4*>(x + k));
          const uint4 w = __ldg(reinterpret_cast<const uint4*>(fr + k));
          const uint32_t hu[4] = {u.x, u.y, u.z, u.w}, hw[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 c = lora_h2f2(hu[j]), e = lora_h2f2(hw[j]);
            s = fmaf(c.x, e.x, s);
            s = fmaf(c.y, e.y, s);
          }
        } else {
          for (int j = k; j < k1; ++j) s = fmaf(lora_h2f(x[j]), lora_h2f(fr[j]), s);
        }
      }
      for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      if (lane == 0) out[r] = r < job.ranks ? scale * s : 0.0f;
    }
    return;
  }
  const int nv = p.R >> 3, step = kThreads / nv;   // k rows per pass
  const int tk = threadIdx.x / nv, v = threadIdx.x - tk * nv;
  float acc[8] = {};
  if (tk < step) {
#pragma unroll 4
    for (int k = k0 + tk; k < k1; k += step) {
      const float xv = lora_h2f(__ldg(x + k));
      const uint4 w =
          __ldg(reinterpret_cast<const uint4*>(f + static_cast<long long>(k) * job.ldf + 8 * v));
      const uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 c = lora_h2f2(h[j]);
        acc[2 * j] = fmaf(xv, c.x, acc[2 * j]);
        acc[2 * j + 1] = fmaf(xv, c.y, acc[2 * j + 1]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) red[threadIdx.x * 9 + j] = acc[j];
  __syncthreads();
  // rank r: the `step` threads' terms in `parts` interleaved groups, then those
  const int parts = kThreads / p.R;
  const int r = threadIdx.x % p.R, part = threadIdx.x / p.R;
  if (part < parts) {
    float s = 0.0f;
    for (int t = part; t < step; t += parts) s += red[(t * nv + (r >> 3)) * 9 + (r & 7)];
    red2[part * p.R + r] = s;
  }
  __syncthreads();
  if (threadIdx.x < p.R) {
    float s = 0.0f;
    for (int t = 0; t < parts; ++t) s += red2[t * p.R + threadIdx.x];
    out[threadIdx.x] = static_cast<int>(threadIdx.x) < job.ranks ? scale * s : 0.0f;
  }
}

struct PackArgs {
  const int* ids;
  const float* part[2];    // [row][slice][r8]
  float* V[2];             // [row][ldv]
  uint16_t* scaled[2];     // may be NULL
  float* unscale[2];
  int M, slices, r8, ldv, chunks;
};

constexpr int kPackThreads = 512;

__global__ void __launch_bounds__(kPackThreads) lora_pack_kernel(const PackArgs p) {
  __shared__ int s_ids[128], s_exp[128];
  __shared__ unsigned int s_top[128];   // by row: largest finite magnitude
  griddep_launch_dependents();
  const int which = blockIdx.y, row0 = blockIdx.x * 128, rows = min(128, p.M - row0);
  const float* const part = (which ? p.part[1] : p.part[0]) +
                            static_cast<long long>(row0) * p.slices * p.r8;
  float* const V = (which ? p.V[1] : p.V[0]) + static_cast<long long>(row0) * p.ldv;
  uint16_t* const scaled = which ? p.scaled[1] : p.scaled[0];
  float* const unscale = (which ? p.unscale[1] : p.unscale[0]) + row0;
  for (int i = threadIdx.x; i < rows; i += kPackThreads) {
    s_ids[i] = __ldg(p.ids + row0 + i);
    s_top[i] = 0u;
  }
  __syncthreads();
  griddep_wait();
  const int per = p.ldv / 4;
  for (int i = threadIdx.x; i < rows * per; i += kPackThreads) {
    const int r = i / per, q = i - r * per;
    const float* src = part + static_cast<long long>(r) * p.slices * p.r8 + 4 * q;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int k = 0; k < p.slices; ++k) {
      const float4 t = __ldcg(reinterpret_cast<const float4*>(src + k * p.r8));
      v.x += t.x;
      v.y += t.y;
      v.z += t.z;
      v.w += t.w;
    }
    reinterpret_cast<float4*>(V)[i] = v;
    if (scaled) atomicMax(s_top + r, lora_top_bits(v));
  }
  if (!scaled) return;
  __syncthreads();
  // a row's scale goes by the largest magnitude of all rows of its adapter here:
  // four threads a row, each a quarter of the rows
  static_assert(kPackThreads == 4 * 128, "four threads a row");
  {
    const int r = threadIdx.x >> 2;
    unsigned int top = 0u;
    if (r < rows)
      for (int i = threadIdx.x & 3; i < rows; i += 4)
        if (s_ids[i] == s_ids[r]) top = max(top, s_top[i]);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    if (r < rows && (threadIdx.x & 3) == 0) {
      s_exp[r] = lora_scale_exponent(__uint_as_float(top));
      unscale[r] = lora_power(-s_exp[r]);
    }
  }
  __syncthreads();
  // eight threads a row and chunk, four ranks each
  const int q = threadIdx.x & 7;
  for (int i = threadIdx.x >> 3; i < rows * p.chunks; i += kPackThreads / 8) {
    const int r = i / p.chunks, c = i - r * p.chunks, piece = 8 * c + q;
    const float4 v = piece < per ? reinterpret_cast<const float4*>(V)[r * per + piece]
                                 : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float up = lora_power(s_exp[r]);
    lora_store_split(scaled + ((static_cast<long long>(row0) + r) * p.chunks + c) * 64 + 4 * q,
                     make_float4(up * v.x, up * v.y, up * v.z, up * v.w));
  }
}

// K slices: about four blocks per SM in all, at least 64 long for the longer job.
int slices_of(const LoraShrinkPlan& p, int sms) {
  const int fill = static_cast<int>(4ll * sms * p.max_c / (p.M * p.sum_c));
  return std::max(1, std::min({kLoraRowSlices, fill, p.max_c / 64}));
}

}  // namespace

cudaError_t launch_lora_rows(const LoraRows& p, cudaStream_t stream) {
  if (p.njobs == 1 && !p.job[0].k_major)
    lora_rows_kernel<true><<<p.M * p.slices, kThreads, 0, stream>>>(p);
  else
    lora_rows_kernel<false><<<p.M * p.slices * p.njobs, kThreads, 0, stream>>>(p);
  return counted_launch(cudaGetLastError());
}

bool lora_rows_suit(const LoraShrinkPlan& p) {
  // the tensor cores' passes: few adapters at a time, an eighth of the k-blocks
  // each, about 0.4 us an iteration; by rows 10 us for 2^25 multiply-adds, so
  // 2^20 multiply-adds take less than an iteration
  const int at_once = p.R <= 16 ? 4 : (p.R <= 32 ? 2 : 1);
  const int most = std::min({p.adapters, p.M, 128});
  const long long iterations = 1ll * ((most + at_once - 1) / at_once) * ((p.max_c + 511) / 512);
  return p.M <= 1024 && iterations >= 24 &&
         p.M * p.sum_c * p.R <= std::min(iterations << 20, 1ll << 26);
}

size_t lora_rows_bytes(const LoraShrinkPlan& p, int sms) {
  const size_t r8 = (p.R + 7) / 8 * 8;
  return lora_shrink_bytes(p) +
         p.njobs * lora_round256(4 * static_cast<size_t>(p.M) * slices_of(p, sms) * r8);
}

int lora_rows(LoraShrinkPlan& p, void* scratch, const LoraDevice& d, cudaStream_t stream) {
  uint8_t* buf = static_cast<uint8_t*>(scratch);
  auto take = [&](size_t bytes) {
    uint8_t* const q = buf;
    buf += lora_round256(bytes);
    return q;
  };
  const int tiles = (p.M + 127) / 128, r8 = (p.R + 7) / 8 * 8;
  LoraRows rows{};
  rows.njobs = p.njobs;
  rows.slices = slices_of(p, d.sms);
  rows.ids = p.ids;
  rows.scales = p.scales;
  rows.M = p.M;
  rows.R = r8;
  rows.adapters = p.adapters;
  PackArgs k{};
  k.ids = p.ids;
  k.M = p.M;
  k.slices = rows.slices;
  k.r8 = r8;
  k.ldv = p.ldv;
  k.chunks = (p.R + 31) / 32;
  for (int j = 0; j < p.njobs; ++j) {
    LoraShrinkJob& job = p.job[j];
    float* const part = reinterpret_cast<float*>(take(4 * static_cast<size_t>(p.M) * rows.slices * r8));
    rows.job[j] = LoraRowsJob{job.x, job.ldx, job.C, job.F, job.ldf, job.f_stride, job.k_major, part,
                              p.R};
    job.V = reinterpret_cast<float*>(take(4 * static_cast<size_t>(p.M) * p.ldv));
    job.tiles = tiles;
    if (job.want & kLoraScaled) {
      job.scaled = reinterpret_cast<uint16_t*>(take(2 * 64 * static_cast<size_t>(k.chunks) * p.M));
      job.unscale = reinterpret_cast<float*>(take(4 * static_cast<size_t>(p.M)));
    }
    k.part[j] = part;
    k.V[j] = job.V;
    k.scaled[j] = job.scaled;
    k.unscale[j] = job.unscale;
  }
  if (launch_lora_rows(rows, stream) != cudaSuccess) return GEMM_ERR_CUDA;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(p.njobs), 1);
  cfg.blockDim = dim3(kPackThreads, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return counted_launch(cudaLaunchKernelEx(&cfg, lora_pack_kernel, k)) == cudaSuccess ? GEMM_OK
                                                                                      : GEMM_ERR_CUDA;
}

}  // namespace gb300
