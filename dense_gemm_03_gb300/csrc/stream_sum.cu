// stream_sum.cu -- adds up the fp32 partial sums of a streamed product (few rows,
// or few tiles with a long K) in chunk order and finishes the result: alpha and
// beta, scales by row and column, a gate, or a gate's gradient.
//
// One block per (row, 128 VEC columns); a thread takes VEC neighbouring columns
// (four, by 16-byte loads, when that still fills the SMs).  Bound by the latency of two
// dependent steps, the stream's end and one round of loads: every chunk's are
// issued before the first is added.
#include "stream_finish.cuh"

namespace gb300 {
namespace {

constexpr int kThreads = 128;

template <int VEC>
__device__ __forceinline__ void load_part(const float* p, float (&v)[VEC]) {
  if constexpr (VEC == 4) {
    const float4 q = __ldcg(reinterpret_cast<const float4*>(p));
    v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
  } else {
    v[0] = __ldcg(p);
  }
}

// The sums of columns c .. c + VEC - 1 of row `row` (columns of the stream; a block's
// last columns may lie past N, inside its unit).
template <int VEC>
__device__ __forceinline__ void add_chunks(const StreamParts& p, int row, int c, float (&s)[VEC]) {
  const int blk = row / p.block;
  const long long step = static_cast<long long>(p.block_rows) * 128;
  const float* src = p.part +
                     (static_cast<long long>(blk) * p.units + (c >> 7)) * p.chunks * step +
                     (row - blk * p.block) * 128 + (c & 127);
#pragma unroll
  for (int i = 0; i < VEC; ++i) s[i] = 0.0f;
  int k = 0;
  for (; k + 8 <= p.chunks; k += 8, src += 8 * step) {
    float v[8][VEC];
#pragma unroll
    for (int u = 0; u < 8; ++u) load_part<VEC>(src + u * step, v[u]);
#pragma unroll
    for (int u = 0; u < 8; ++u)
#pragma unroll
      for (int i = 0; i < VEC; ++i) s[i] += v[u][i];
  }
  float v[7][VEC];
#pragma unroll
  for (int u = 0; u < 7; ++u)
    if (k + u < p.chunks) load_part<VEC>(src + u * step, v[u]);
#pragma unroll
  for (int u = 0; u < 7; ++u)
    if (k + u < p.chunks)
#pragma unroll
      for (int i = 0; i < VEC; ++i) s[i] += v[u][i];
}

// vec: the results' rows (and dC's) are on the grid of VEC elements.
template <int GATE, bool F32, bool SCALED, int VEC>
__global__ void __launch_bounds__(kThreads) stream_sum_kernel(const StreamSum p, bool vec) {
  griddep_launch_dependents();
  const int strips = (p.N + kThreads * VEC - 1) / (kThreads * VEC);
  const int row = blockIdx.x / strips;
  const int c = ((blockIdx.x - row * strips) * kThreads + static_cast<int>(threadIdx.x)) * VEC;
  const int n = min(VEC, p.N - c);   // columns that exist
  griddep_wait();
  if (n <= 0) return;
  const bool v = vec && n == VEC;
  float s[VEC], u[VEC];
  add_chunks<VEC>(p.parts, row, c, s);
  if constexpr (GATE != 0) add_chunks<VEC>(p.parts, row, p.N + c, u);
  stream_finish<GATE, F32, SCALED, VEC>(p, row, c, n, v, s, u);
}

template <int GATE, bool F32, bool SCALED>
cudaError_t launch(const StreamSum& s, const LoraDevice& d, cudaStream_t stream) {
  // four columns a thread where that still gives the SMs a block each, and where U's
  // columns lie on the same grid as G's
  const long long strips4 = (s.N + 4 * kThreads - 1) / (4 * kThreads);
  const bool wide = s.M * strips4 >= d.sms && (GATE == 0 || s.N % 4 == 0);
  const long long strips = wide ? strips4 : (s.N + kThreads - 1) / kThreads;
  const long long blocks = s.M * strips;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  const uintptr_t elem = F32 ? 16 : 8;
  uintptr_t bits = reinterpret_cast<uintptr_t>(s.C);
  bool vec = s.ldc % 4 == 0;
  if (GATE == 2) {
    bits |= reinterpret_cast<uintptr_t>(s.g.dC) | reinterpret_cast<uintptr_t>(s.g.dU);
    vec = vec && s.g.lddc % 4 == 0;
  }
  vec = vec && bits % elem == 0;
  const unsigned grid = static_cast<unsigned>(blocks);
  return wide ? launch_early(stream_sum_kernel<GATE, F32, SCALED, 4>, grid, kThreads, 0, stream, s, vec)
              : launch_early(stream_sum_kernel<GATE, F32, SCALED, 1>, grid, kThreads, 0, stream, s, vec);
}

}  // namespace

int stream_sum(const StreamSum& s, const LoraDevice& d, cudaStream_t stream) {
  cudaError_t e = cudaErrorInvalidValue;
  if (s.gate == 0)
    e = s.scaled ? launch<0, false, true>(s, d, stream)
        : s.f32  ? launch<0, true, false>(s, d, stream)
                 : launch<0, false, false>(s, d, stream);
  else if (s.gate == 1)
    e = s.scaled ? launch<1, false, true>(s, d, stream) : launch<1, false, false>(s, d, stream);
  else if (!s.scaled)
    e = launch<2, false, false>(s, d, stream);
  return counted_launch(e) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

}  // namespace gb300
