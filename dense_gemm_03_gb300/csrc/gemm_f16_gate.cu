// gemm_f16_gate.cu -- launchers of the tcgen05 half-precision GEMM kernel
// (gemm_f16_tc_kernel.cuh) on CTA pairs with gated results, their gradient, and
// results scaled by row and column.
#include "gemm_f16_tc_kernel.cuh"

namespace gb300 {
namespace {

template <int GATE, bool SCALED, bool FOLD = false>
cudaError_t launch(int epi, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& c,
                   const CUtensorMap& u, const GateArgs& gate, const TcArgs& args, int grid,
                   cudaStream_t s) {
  using G = Gated<GATE, SCALED, FOLD>;
  G x{};
  x.tmU = u;
  x.a = gate;
  if (epi == kEpiTma)
    return launch_one<256, kLoadTma, kEpiTma, true, 128, 128, 1, G>(a, b, c, args, grid, s, x);
  // (a plain product's C off the 16-byte grid is written by way of an aligned copy)
  if constexpr (GATE != 0)
    if (epi == kEpiManual)
      return launch_one<256, kLoadTma, kEpiManual, true, 128, 128, 1, G>(a, b, c, args, grid, s, x);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_gemm_f16_tc_gate(int gate, bool scaled, bool fold, int epi_mode, const CUtensorMap& tmA,
                                    const CUtensorMap& tmB, const CUtensorMap& tmC,
                                    const CUtensorMap& tmU, const GateArgs& gate_args,
                                    const TcArgs& args, int grid, cudaStream_t stream) {
  switch (gate) {
    case 0:
      return scaled ? launch<0, true>(epi_mode, tmA, tmB, tmC, tmU, gate_args, args, grid, stream)
                    : cudaErrorInvalidValue;
    case 1:
      return scaled ? launch<1, true>(epi_mode, tmA, tmB, tmC, tmU, gate_args, args, grid, stream)
                    : launch<1, false>(epi_mode, tmA, tmB, tmC, tmU, gate_args, args, grid, stream);
    default:
      return scaled ? cudaErrorInvalidValue
             : fold ? launch<2, false, true>(epi_mode, tmA, tmB, tmC, tmU, gate_args, args, grid, stream)
                    : launch<2, false>(epi_mode, tmA, tmB, tmC, tmU, gate_args, args, grid, stream);
  }
}

}  // namespace gb300
