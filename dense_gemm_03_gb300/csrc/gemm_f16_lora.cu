// gemm_f16_lora.cu -- launchers of the tcgen05 half-precision GEMM kernel
// (gemm_f16_tc_kernel.cuh) with low-rank adapters picked by row as more
// k-blocks of its tiles: CTA pairs, B as it is or transposed.
#include "gemm_f16_tc_kernel.cuh"

namespace gb300 {
namespace {

template <bool TRANS>
cudaError_t launch(int epi, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& c,
                   const CUtensorMap& e, const CUtensorMap& v, const LoraTailArgs& tail,
                   const TcArgs& args, int grid, cudaStream_t s) {
  LoraTail<TRANS> x{};
  x.tmE = e;
  x.tmV = v;
  x.a = tail;
  return epi == kEpiTma
             ? launch_one<256, kLoadTma, kEpiTma, true, 128, 128, 1, LoraTail<TRANS>>(a, b, c, args,
                                                                                     grid, s, x)
             : cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_gemm_f16_tc_lora(bool trans, int epi_mode, const CUtensorMap& tmA,
                                    const CUtensorMap& tmB, const CUtensorMap& tmC,
                                    const CUtensorMap& tmE, const CUtensorMap& tmV,
                                    const LoraTailArgs& tail,
                                    const TcArgs& args, int grid, cudaStream_t stream) {
  return trans ? launch<true>(epi_mode, tmA, tmB, tmC, tmE, tmV, tail, args, grid, stream)
               : launch<false>(epi_mode, tmA, tmB, tmC, tmE, tmV, tail, args, grid, stream);
}

}  // namespace gb300
