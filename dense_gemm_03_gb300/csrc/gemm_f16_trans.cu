// gemm_f16_trans.cu -- launchers of the tcgen05 half-precision GEMM kernel
// (gemm_f16_tc_kernel.cuh) on CTA pairs with operands stored transposed, half
// and float C.
#include "gemm_f16_tc_kernel.cuh"

namespace gb300 {
namespace {

template <bool TA, bool TB>
cudaError_t launch(int epi, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& c,
                   const TcArgs& args, int grid, cudaStream_t s) {
  using T = Transposed<TA, TB, false>;
  using F = Transposed<TA, TB, true>;
  F fold;
  fold.fold_kb = args.kb_total >= 64 ? 16 : 8;
  switch (epi) {
    case kEpiTma:
      return launch_one<256, kLoadTma, kEpiTma, true, 128, 128, 1, T>(a, b, c, args, grid, s);
    case kEpiF32Tma:
      return launch_one<256, kLoadTma, kEpiF32Tma, true, 128, 128, 1, F>(a, b, c, args, grid, s, fold);
    case kEpiF32:
      return launch_one<256, kLoadTma, kEpiF32, true, 128, 128, 1, F>(a, b, c, args, grid, s, fold);
    default:
      return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_gemm_f16_tc_trans(bool trans_a, bool trans_b, int epi_mode,
                                     const CUtensorMap& tmA, const CUtensorMap& tmB,
                                     const CUtensorMap& tmC, const TcArgs& args, int grid,
                                     cudaStream_t stream) {
  if (trans_a)
    return trans_b ? launch<true, true>(epi_mode, tmA, tmB, tmC, args, grid, stream)
                   : launch<true, false>(epi_mode, tmA, tmB, tmC, args, grid, stream);
  return trans_b ? launch<false, true>(epi_mode, tmA, tmB, tmC, args, grid, stream)
                 : cudaErrorInvalidValue;
}

}  // namespace gb300
